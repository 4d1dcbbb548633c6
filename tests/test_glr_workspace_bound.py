"""The bound that include/lt2_gdr.h gives for the gated linear recurrence's scratch holds at every size."""
import itertools
import random

import pytest

import gated_delta_rule_looped_b200 as lt2
from gated_delta_rule_looped_b200 import build as lbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    if lbuild.needs_build():
        lbuild.build()


def bound(units, L, d):
    return 12 * units * -(-L // 64) * -(-d // 64) * 64 + 512


def sizes():
    yield from itertools.product((1, 3, 37, 500), (1, 2, 9, 33, 64, 65, 129, 1000, 65536), (1, 3, 16, 17, 24, 32, 33, 64, 65, 128, 130, 2560))
    r = random.Random(1)
    for _ in range(3000):
        yield int(2 ** r.uniform(0, 12)), int(2 ** r.uniform(0, 18)), int(2 ** r.uniform(0, 12))


def test_scratch_stays_within_the_bound():
    most = 0.0
    for units, L, d in sizes():
        dims = lt2.lt2_glr_dims(1, units, 1, L, d, 1, 1, 1, 0.5, 0, 0)
        n = lt2.lt2_glr_prefill_workspace_bytes(dims)
        assert n <= bound(units, L, d), (units, L, d, n)
        most = max(most, n / bound(units, L, d))
        # the backward pass adds the states that it may have to compute again
        b = lt2.lt2_glr_backward_workspace_bytes(dims)
        assert b <= bound(units, L, d) + 4 * units * -(-L // 64) * d, (units, L, d, b)
    assert most > 0.9                                          # and is not far above it

