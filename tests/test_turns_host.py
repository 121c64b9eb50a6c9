"""The rotation's 128-bit turn fractions (csrc/turns.h) against wide integers, compiled for the host."""
import os
import shutil
import subprocess

import pytest

from tests.wide_turns import BITS, turns

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_long_sequence_gb300", "csrc")
MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "turns.h"
int main(int argc, char** argv) {
    for (int k = 1; k < argc; ++k)
        for (int rot = 16; rot <= 64; rot += 16) {
            uint64_t hi[32], lo[32];
            dfs::turns::fill(hi, lo, std::strtod(argv[k], nullptr), rot);
            for (int i = 0; i < rot / 2; ++i)
                std::printf("%d %d %d %llx %llx\n", k, rot, i, (unsigned long long)hi[i], (unsigned long long)lo[i]);
        }
}
"""
THETAS = [1.0, float.fromhex("0x1.0000000000001p+0"), 1.5, 2.0, 3.7, 10000.0, 500000.0, 1e6, 1.0e15, 12345.678901234567, 1e100,
          1e300, 1.7976931348623157e308]


def test_fractions(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "turns.cpp", tmp_path / "turns"
    src.write_text(MAIN)
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe), *(t.hex() for t in THETAS)], check=True, capture_output=True, text=True).stdout
    lines = out.splitlines()
    assert len(lines) == len(THETAS) * (8 + 16 + 24 + 32)
    for line in lines:
        k, rot, i, hi, lo = line.split()
        theta, want = THETAS[int(k) - 1], turns(THETAS[int(k) - 1], int(rot))[int(i)]
        got = ((int(hi, 16) << 64) | int(lo, 16)) << (BITS - 128)
        # 2^-120 of the fraction and the last place
        assert abs(got - want) <= (want >> 120) + (1 << (BITS - 128)), (theta, rot, i)
