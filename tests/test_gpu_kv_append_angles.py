"""The cosines and sines of lt2_kv_append are those of the exact angle, rounded once, at every position.

Rows of (1, 0) pairs come out as (cos, sin): the products with 1 and 0 and their sum are exact.  Tolerance, from the arithmetic:
the angle is a whole number of 2^-64 turns a position, off by less than three (the quotient's two roundings in 64 bits, and
the cut), so position p is off by less than 3 p 2^-64 turns, 6 pi p 2^-64 in the value; as a double in half turns by 2^-53
relative, pi 2^-53; its sine and cosine by a few units of 2^-53; then one rounding to fp32, 2^-24 of the value at most.  With p
below 2^21 all but the last are below 2^-38.
"""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import gated_delta_rule_looped_b200 as lt2
from tests.gpu_util import to_np

pytestmark = pytest.mark.gpu


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def exact(pos, freq):
    """cos and sin of pos * freq, whole turns taken off in integers of 2^-80 turns."""
    turns = [math.floor(Fraction(f) / (2 * PI) * 2 ** 80) for f in freq]
    ang = np.array([[(int(p) * t % (1 << 80)) / 2.0 ** 80 for t in turns] for p in pos])
    # the nearest quarter turn off, so that a double holds the rest to all its bits
    q = np.round(ang * 4)
    rest = 2 * math.pi * (ang - q / 4)
    c, s, q = np.cos(rest), np.sin(rest), q.astype(int) % 4
    return np.choose(q, [c, -s, -c, s]), np.choose(q, [s, c, -s, -c])


def frequencies(rot):
    """base^(-2 i / rot), and some beside a half and a whole turn a token."""
    f = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    f[1], f[2], f[3], f[4] = math.pi * (1 - 2.0 ** -20), math.pi * (2 - 2.0 ** -18), 1e-7, -math.pi / 2
    return f


@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (128, 64, True), (12, 12, False), (33, 32, False), (36, 26, True)])
@pytest.mark.parametrize("first", [0, 1 << 20])
def test_cosines_and_sines_are_rounded_once(d, rot, interleaved, first):
    n, f = 500, frequencies(rot)
    i0 = np.arange(rot // 2) * 2 if interleaved else np.arange(rot // 2)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    q = torch.zeros((1, 1, n, d), device="cuda")
    q[..., i0] = 1.0
    k, pages = torch.zeros_like(q), (first + n) // 64 + 1
    kc, vc = (torch.zeros((1, 9, 1, 64, d), device="cuda") for _ in range(2))
    table = (torch.arange(pages, device="cuda", dtype=torch.int32) % 9)[None].contiguous()
    out, _ = lt2.kv_append(q, k, k.clone(), kc, vc, table, torch.tensor([first], device="cuda"),
                           cu_seqlens=torch.tensor([0, n], device="cuda"), rope=lt2.make_rope(rot, interleaved=interleaved, inv_freq=f))
    assert lt2.lt2_gdr_last_device_error() == lt2.LT2_OK
    c, s = exact(range(first, first + n), f)
    got = to_np(out)[0, 0]
    for name, g, ref in (("cos", got[:, i0], c), ("sin", got[:, i1], s)):
        err = np.abs(g - ref)
        assert (err <= 2.0 ** -24 * np.abs(ref) + 2.0 ** -38).all(), (name, (err / (np.abs(ref) + 2.0 ** -16)).max() * 2 ** 24)
