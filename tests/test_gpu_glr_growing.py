"""The gated linear recurrence with decays above one over thousands of tokens: their product over 64 tokens is finite, over all
of them it is not, and the states stay finite because nothing is written meanwhile.

Tolerances: those of tests/test_gpu_glr.py, whose bounds hold for any decay.
"""
import math

import pytest
import torch

import gated_delta_rule_looped_b200 as lt2
from tests.test_gpu_glr import backward, check_backward, check_forward, forward, make

pytestmark = pytest.mark.gpu


def growing(T, B, H, L, d, xt, gt, seed):
    """An ordinary stretch, a reset, a stretch of zeros that grows by `up` a token, a reset, and an ordinary stretch again."""
    v = make(T, B, H, L, d, xt, gt, False, True, True, seed)
    a, b = L // 8, L - L // 8
    up = 2.5
    assert 64 * math.log2(up) < 127 and (b - a) * math.log2(up) > 128
    for n in ("x", "dO"):
        v[n][..., a:b, :] = 0
    v["a"][..., a:b, :] = up
    v["a"][..., a, :] = 0                                      # the states before do not grow
    v["a"][..., b, :] = 0                                      # nor, backward, the gradients behind
    return v


# narrow units (in segments), a few channels (tiles that wait for one another), many channels (streamed): 64 and 32 to a chain
SHAPES = [(1, 2, 1, 4099, 4), (2, 1, 2, 2500, 15), (1, 1, 3, 20000, 1), (1, 1, 2, 2049, 128), (1, 2, 1, 1000, 36),
          (3, 5, 11, 700, 130), (1, 4, 37, 1030, 32), (1, 2, 2, 300, 20)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16")])
def test_states_that_stay_finite_between_growing_decays(shape, types):
    v = growing(*shape, *types, seed=sum(shape))
    o, S, states = forward(v, save_states=True)
    g = backward(v, states=states)
    g2 = backward(v)
    # zeros are zeros, whatever they are multiplied by
    a, b = shape[3] // 8, shape[3] - shape[3] // 8
    assert not o[..., a:b, :].any() and not g["dx"][..., a + 1:b, :].any()
    some = (lambda t: t[:, :, ::5].contiguous() if isinstance(t, torch.Tensor) else t) if shape[2] > 5 else (lambda t: t)
    part = {n: some(t) for n, t in v.items()}
    check_forward(part, some(o), some(S), some(states))
    check_backward(part, {n: some(t) for n, t in g.items()})
    assert all(torch.equal(g[n], g2[n]) for n in g)
    assert lt2.lt2_gdr_last_device_error() == lt2.LT2_OK
