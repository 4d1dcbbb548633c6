"""Keys of a page outside the cache are left out of the decode attention (lt2_swa_decode): the results are those of the keys that
remain, not of zeros in their place.

Tolerances: those of tests/test_gpu_swa_decode.py, with weights of 24 bits.
"""
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_looped_b200 as lt2
from tests.gpu_util import to_np
from tests.test_gpu_swa_decode import ALL, CC, U, run, setup

pytestmark = pytest.mark.gpu


def reference(s, gone):
    """o without the table columns `gone[b]` of sequence b, sum_s p_s |v_s|, the largest sum |q k| scale of a row, and what comes out
    if their keys count as zeros."""
    q, kc, vc, table = (to_np(s[n]) for n in ("q", "kc", "vc", "table"))
    T, B, Hq, d = q.shape
    size, Hkv = kc.shape[3], kc.shape[2]
    o, A, D, zeros = np.zeros(q.shape), np.zeros(q.shape), np.zeros((T, B, Hq, 1)), np.zeros(q.shape)
    for b, n in enumerate(s["lens"]):
        pos = np.arange(max(0, n - s["window"]), n)
        if not len(pos):
            continue
        here = ~np.isin(pos // size, gone[b])
        pages = np.where(here, table[b].astype(int)[pos // size], 0)
        for h in range(Hq):
            k, v = (np.where(here[:, None], c[:, pages, h // (Hq // Hkv), pos % size], 0.0) for c in (kc, vc))
            x = np.einsum("td,tnd->tn", q[:, b, h], k) / math.sqrt(d)
            D[:, b, h, 0] = np.einsum("td,tnd->tn", np.abs(q[:, b, h]), np.abs(k)).max(1) / math.sqrt(d)
            for count, out in ((here, o), (np.ones_like(here), zeros)):
                if not count.any():
                    continue
                w = np.where(count, np.exp(x - x.max(1, keepdims=True)), 0.0)
                out[:, b, h] = np.einsum("tn,tnd->td", w, v) / w.sum(1)[:, None]
                if out is o:
                    A[:, b, h] = np.einsum("tn,tnd->td", w, np.abs(v)) / w.sum(1)[:, None]
    return o, A, D, zeros


def check(s, gone, algo=lt2.LT2_ALGO_AUTO, tell=True):
    d = s["q"].shape[-1]
    ref, A, D, zeros = reference(s, gone)
    tc = s["q"].dtype == torch.bfloat16 and d % 8 == 0 and algo != CC
    e = ((d + 15) // 16 * 2.0 ** -22 if tc else 14 * U) * D + 3 * U * D
    tol = A * (2 * (e + 2.0 ** -22) + (max(s["lens"]) / 16 + 32) * 2.0 ** -22) + U * np.abs(ref)
    if tell:                                                   # the tolerance tells the two apart
        assert (np.abs(zeros - ref) > 10 * tol).any()
    # pages that no window reaches are not looked at
    seen = any(c in np.arange(max(0, n - s["window"]), n) // s["kc"].shape[3] for n, cols in zip(s["lens"], gone) for c in cols)
    for page in (-1, s["kc"].shape[1], 1 << 30):
        bad = dict(s, table=s["table"].clone())
        for b, cols in enumerate(gone):
            bad["table"][b, list(cols)] = page
        o = to_np(run(bad, algo, out="f32"))
        assert lt2.lt2_gdr_last_device_error() == (lt2.LT2_ERR_PAGES if seen else lt2.LT2_OK)
        out = ~(np.abs(o - ref) <= tol)
        assert not out.any(), f"{out.sum()} of {out.size} out, worst {np.nanmax(np.abs(o - ref) / (tol + 1e-30)):.1f} times the bound"
    assert lt2.lt2_gdr_last_device_error() == lt2.LT2_OK


# (T, Hq, Hkv, d, page size): few CTAs (many warps each) and many, both halves of the rows, both ring depths, a page of one tile and
# of several
HEADS = [(1, 2, 1, 128, 16), (1, 34, 2, 64, 64), (1, 4, 2, 256, 16), (2, 60, 30, 128, 16), (2, 60, 30, 64, 32), (1, 3, 3, 72, 256),
         (2, 72, 6, 128, 64)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("dtype,algo", [("bf16", lt2.LT2_ALGO_AUTO), ("bf16", CC), ("f32", lt2.LT2_ALGO_AUTO)])
@pytest.mark.parametrize("window", [ALL, 300])
def test_own_keys(heads, dtype, algo, window):
    s = setup(*heads, [700, 33, 0, 520], window, dtype, seed=heads[3])
    size = heads[4]
    last = lambda n: (n - 1) // size
    # the last page of each, one in the middle, two in a row at the end, the window's first
    check(s, [[last(700)], [], [], [last(520), last(520) - 1]], algo)
    check(s, [[500 // size, 650 // size], [0], [], [max(0, 520 - window) // size]], algo)


@pytest.mark.parametrize("size", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 2, 2), (2, 12, 2), (1, 40, 2)])
@pytest.mark.parametrize("window", [ALL, 900])
def test_shared_prefix(size, heads, window):
    prefix = 1024
    s = setup(*heads, 128, size, [1100, 1025, 0, 1300, 1031], window, "bf16", seed=size, prefix=prefix)
    n = prefix // size
    for cols in ([0], [n // 2], [n - 1], [n // 2 - 1, n // 2, n - 1], [600 // size, 700 // size]):
        check(s, [cols if k else [] for k in s["lens"]], tell=cols != [0] or window == ALL or size == 256)
    # a page of the shared part and one of a sequence's own
    check(s, [[n // 2], [n // 2], [], [n // 2, 1299 // size], [n // 2]])


def test_nothing_remains():
    """Every page of a sequence is bad: zeros, as without keys."""
    for heads, prefix in (((1, 2, 1, 128, 64), 0), ((1, 4, 2, 128, 64), 512)):
        s = setup(*heads, [512, 600], ALL, "bf16", seed=3, prefix=prefix)
        s["table"][:, : 512 // 64] = -1
        o = run(s)
        assert lt2.lt2_gdr_last_device_error() == lt2.LT2_ERR_PAGES
        assert not o[:, 0].any() and o[:, 1].any()
