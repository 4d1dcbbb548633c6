"""Numbers past the width of their field in the C ABI: ctypes cuts them without a word, so the binding must not hand them on."""
import pytest
import torch

import gated_delta_rule_looped_b200 as lt2


@pytest.mark.parametrize("rot", [1 << 31, (1 << 32) + 64, -(1 << 32) + 64])
def test_a_rotation_wider_than_its_field_is_refused(rot):
    with pytest.raises(ValueError):
        lt2.make_rope(rot)
    assert lt2.make_rope((1 << 31) - 2).rot_dim == (1 << 31) - 2       # the call itself refuses what no row holds


def _decode(window=None, prefix_len=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q, k, v = (torch.randn(n, generator=g, device="cuda").to(torch.bfloat16) for n in ((1, 2, 1, 64), (1, 2, 1, 16, 64), (1, 2, 1, 16, 64)))
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    return lt2.swa_decode(q, k, v, table, torch.tensor([16, 9], device="cuda"),
                          window=window, prefix_len=prefix_len)


@pytest.mark.gpu
def test_a_window_wider_than_its_field_sees_everything():
    ref = _decode()
    for w in (1 << 62, 1 << 63, (1 << 64) + 1, (1 << 64) + 5, 10 ** 30):
        assert torch.equal(_decode(window=w), ref)
    assert not torch.equal(_decode(window=5), ref)


@pytest.mark.gpu
def test_negative_numbers_are_refused_whatever_their_size():
    for n in (-1, -(1 << 63) - 5, -(1 << 64) + 5, -10 ** 30):
        with pytest.raises(lt2.Lt2Error):
            _decode(window=n)
        with pytest.raises(lt2.Lt2Error):
            _decode(prefix_len=n)
