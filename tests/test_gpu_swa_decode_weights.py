"""The softmax weights of bf16 decode attention (lt2_swa_decode) keep all 24 bits of fp32 on their way into the
product with the values.

Every value is zero but for one column, so that an output is the sum of the few weights of its column over the sum of all.
Tolerance, from the arithmetic (u = 2^-24, s a step of 2^-22 that the tensor core's accumulation takes at most), with D the
largest sum_i |q_i k_i| scale, n keys, and k of them in a column: a score is off by e = d / 16 s D + 3 u D, exp2 by s
relative, so a weight by w = e + s, in the sum of all weights too.  A column accumulates three exact parts of a bf16 x bf16
product for each of its keys, 3 k s; the sum of all weights takes two additions for 16 keys in a lane, then three exchanges
and at most 16 warps, (n / 8 + 20) u; joining warps and splits multiplies and adds, 2 x (16 + splits) u and an exp2 of s
each, the last division 2 u.  Each of these steps is relative to partial sums that are no larger than A = sum_s p_s |v_s| of the column
(the values of one column differ in sign, so its sum may be smaller), so the output is off by A times 2 w + (3 k + 2) s +
(n / 8 + 2 splits + 54) u.  The inputs have D below 1/2, where that is 2^-17 A for 100 keys: weights of 16 bits miss it.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_looped_b200 as lt2
from oracle import cache
from tests.gpu_util import to_np
from tests.test_gpu_swa_decode import ALL, setup

pytestmark = pytest.mark.gpu

U, STEP = 2.0 ** -24, 2.0 ** -22
SPLITS = 6                                                     # at the lengths below: 512 keys to a split, four blocks of a prefix


def one_column_each(s, seed):
    """Values of one entry, 1 to 2 in size, in the column of their place in the cache; scores near zero."""
    T, pages, H, size, d = s["vc"].shape
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    v = torch.rand((T, pages, H, size, 1), generator=g, device="cuda") + 1
    v *= torch.randint(0, 2, v.shape, generator=g, device="cuda") * 2 - 1
    # consecutive positions take consecutive columns, page by page of the sequences
    col = torch.zeros((pages, size), dtype=torch.long, device="cuda")
    table = to_np(s["table"]).astype(int)
    for b, n in enumerate(s["lens"]):
        for p in range((n + size - 1) // size):
            col[table[b, p]] = torch.arange(p * size, (p + 1) * size, device="cuda") % d
    hot = torch.nn.functional.one_hot(col, d).bool()[None, :, None]
    keep = s["vc"].isnan()
    s["vc"] = torch.where(hot, v, torch.zeros_like(v)).to(torch.bfloat16)
    s["vc"][keep] = float("nan")
    s["q"] = (s["q"] / 32).contiguous()
    return s


def check(s):
    ref, A, D = cache.decode(*(to_np(s[n]) for n in ("q", "kc", "vc")), to_np(s["table"]).astype(int), s["lens"], s["window"])
    d, n = s["q"].shape[-1], min(max(s["lens"]), s["window"])
    assert D.max() < 0.5
    k = -(-n // d)
    w = (d / 16 * STEP + 3 * U) * D + STEP
    rel = 2 * w + (3 * k + 2) * STEP + (n / 8 + 2 * SPLITS + 54) * U
    o = to_np(lt2.swa_decode(s["q"], s["kc"], s["vc"], s["table"], s["n"], window=None if s["window"] == ALL else s["window"],
                             prefix_len=s["prefix"], out="f32"))
    bad = ~(np.abs(o - ref) <= rel * A + U * np.abs(ref))
    assert not bad.any(), f"{bad.sum()} of {bad.size} out, by {np.nanmax(np.abs(o - ref) / (A + 1e-30)):.2e} of {rel.max():.2e}"
    assert lt2.lt2_gdr_last_device_error() == lt2.LT2_OK


@pytest.mark.parametrize("heads", [(1, 2, 2, 128, 16), (2, 34, 2, 64, 32), (1, 4, 1, 256, 64), (1, 2, 1, 72, 128), (2, 60, 30, 128, 32)])
@pytest.mark.parametrize("lens,window", [([3, 64, 0, 100], ALL), ([300, 17], 50), ([1, 130], ALL)])
def test_weights(heads, lens, window):
    check(one_column_each(setup(*heads, lens, window, "bf16", seed=heads[3] + len(lens)), 1))


@pytest.mark.parametrize("heads", [(1, 2, 2, 128, 16), (2, 4, 1, 128, 64), (1, 12, 2, 128, 256)])
@pytest.mark.parametrize("lens,window", [([260, 300, 257], ALL), ([520, 513, 0, 530], ALL), ([520, 525], 400)])
def test_weights_of_a_shared_prefix(heads, lens, window):
    prefix = min(n for n in lens if n) // 256 * 256
    check(one_column_each(setup(*heads, lens, window, "bf16", seed=heads[4], prefix=prefix), 2))
