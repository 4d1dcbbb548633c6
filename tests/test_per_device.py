"""What the library keeps for a GPU is kept apart for every GPU (csrc/per_device.h)."""
import subprocess

from gated_delta_rule_looped_b200 import build as lbuild

PROGRAM = r"""
#include <cstdio>
#include "per_device.h"
int main()
{
    static lt2::PerDevice kept;
    int asked = 0;
    auto of = [&](int dev, int n) { return kept.get(dev, [&]() { ++asked; return n; }); };
    auto show = [&](int dev, int n) { std::printf("%d ", of(dev, n)); };
    // two GPUs of different sizes, each asked for once
    show(0, 296);
    show(1, 264);
    show(0, 1);
    show(1, 1);
    std::printf("%d ", asked);
    // a failure is not kept, nor what belongs to a device past the table or to none
    show(2, 0);
    show(2, 148);
    show(64, 7);
    show(64, 8);
    show(-1, 9);
}
"""


def test_a_number_is_kept_for_each_device(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", f"-I{lbuild.CSRC}", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert out.split() == ["296", "264", "296", "264", "2", "0", "148", "7", "8", "9"]

