"""lt2_kv_append refuses rotations and rows wider than its tables before it writes a frequency anywhere.  Each call is made
in a process of its own: a write past a table on the host's stack would end it."""
import subprocess
import sys

import pytest

import gated_delta_rule_looped_b200 as lt2
from gated_delta_rule_looped_b200 import build as lbuild
from tests.conftest import ROOT

CALLS = """
import gated_delta_rule_looped_b200 as lt2
from tests.test_abi_cache import append, kv_dims
d, rot, given = {d}, {rot}, {given}
rope = lt2.make_rope(rot, inv_freq=[0.5] * (rot // 2) if given else None)
print(append(kv_dims(T=1, Hq=1, Hkv=1, d=d), rope))
# an ordinary call behind it gets as far as the device's checks
print(append(rope=lt2.make_rope(64)))
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    if lbuild.needs_build():
        lbuild.build()


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("d,rot", [(257, 256), (258, 258), (288, 288), (512, 512), (512, 64), (65536, 65536)])
def test_wide_rotations_are_refused(d, rot, given):
    r = subprocess.run([sys.executable, "-c", CALLS.format(d=d, rot=rot, given=given)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    first, second = (int(x) for x in r.stdout.split())
    assert first == lt2.LT2_ERR_UNSUPPORTED
    assert second in (lt2.LT2_ERR_CUDA, lt2.LT2_ERR_INVALID_ARGUMENT)  # no device, or addresses that no device knows


def test_the_widest_rotation_is_taken():
    from tests.test_abi_cache import append, kv_dims
    st = append(kv_dims(T=1, Hq=1, Hkv=1, d=256), lt2.make_rope(256))
    assert st in (lt2.LT2_ERR_CUDA, lt2.LT2_ERR_INVALID_ARGUMENT)
