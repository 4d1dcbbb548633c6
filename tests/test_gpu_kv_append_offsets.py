"""Appending with bad packed offsets (lt2_kv_append): LT2_ERR_SEQLENS is recorded, the sequences of a bad offset leave every
output as it was, and the others arrive as they do under good offsets."""
import pytest
import torch

import gated_delta_rule_looped_b200 as lt2
from tests.test_gpu_kv_append import setup

pytestmark = pytest.mark.gpu

LOW, HIGH = -(1 << 63), (1 << 63) - 1
# (offsets of five sequences over 23 packed tokens, the sequences that must arrive)
CASES = [([-3, 5, 10, 20, 22, 23], [1, 2, 3, 4]), ([LOW, 5, 10, 20, 22, 23], [1, 2, 3, 4]), ([LOW, LOW, 10, 20, 22, 23], [2, 3, 4]),
         ([LOW, LOW, LOW, LOW, LOW, LOW], []), ([-1, -1, -1, -1, -1, 23], []),
         ([0, 5, 10, 20, 22, 1 << 40], [0, 1, 2, 3]), ([0, 5, 10, 20, HIGH, HIGH], [0, 1, 2]), ([0, 5, 10, 20, 22, 24], [0, 1, 2, 3]),
         ([HIGH, HIGH, HIGH, HIGH, HIGH, HIGH], []), ([0, 9, 4, 20, 22, 23], [3, 4]), ([0, 5, 3, 8, 21, 23], [3, 4]),
         ([0, 5, 10, 20, 22, 7], [0, 1, 2]), ([23, 20, 15, 10, 5, 0], []), ([4, LOW, 10, 20, 22, 23], [2, 3, 4]),
         ([0, 5, -2, 20, 22, 23], [3, 4])]


@pytest.mark.parametrize("cu,arrive", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_sequences_of_bad_offsets_are_left_unwritten(cu, arrive, interleaved):
    rope = lt2.make_rope(64, interleaved=interleaved)
    s = setup(2, 2, 1, 64, 16, [4, 40, 0, 17, 300], [5, 5, 5, 5, 3], "bf16", seed=8)
    # every position of every sequence has a page of its own, so that whatever is written shows
    width = s["table"].shape[1]
    s["table"] = torch.arange(5 * width, device="cuda", dtype=torch.int32).view(5, width)
    for n in ("kc", "vc"):
        s[n] = torch.full((2, 5 * width, 1, 16, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    n = s["q"].shape[2]
    assert n == 23 + 3
    for t in ("q", "k", "v"):
        s[t] = s[t][:, :, :23].contiguous()
    s["cu"] = torch.tensor(cu, dtype=torch.int64, device="cuda")
    outs = {"kc": s["kc"], "vc": s["vc"], "q": torch.full_like(s["q"], 7.0), "k": torch.full_like(s["k"], 7.0)}
    lt2.kv_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["table"], s["start"], cu_seqlens=s["cu"], rope=rope,
                  q_out=outs["q"], k_out=outs["k"])
    assert lt2.lt2_gdr_last_device_error() == lt2.LT2_ERR_SEQLENS
    # the sequences that must arrive, one by one by themselves
    want = {t: torch.full_like(x, 7.0) for t, x in outs.items()}
    for b in arrive:
        rows = slice(cu[b], cu[b + 1])
        part = {t: s[t][:, :, rows].contiguous() for t in ("q", "k", "v")}
        one = torch.tensor([0, cu[b + 1] - cu[b]], dtype=torch.int64, device="cuda")
        q, k = lt2.kv_append(part["q"], part["k"], part["v"], want["kc"], want["vc"], s["table"][b:b + 1].contiguous(),
                             s["start"][b:b + 1].contiguous(), cu_seqlens=one, rope=rope, k_out=True)
        want["q"][:, :, rows], want["k"][:, :, rows] = q, k
    assert lt2.lt2_gdr_last_device_error() == lt2.LT2_OK
    for t in outs:
        assert torch.equal(outs[t], want[t]), t
