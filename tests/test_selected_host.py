"""Host-side refusals of the rotation alone and of the attention over chosen key blocks: every
argument check answers before anything touches a device (no compute call is made here); the
rotation's turn fractions of given frequencies against wide integers; warps meet before warp-wide
instructions."""
import ctypes
import glob
import os
import re
import shutil
import subprocess
from fractions import Fraction

import pytest

from sparse_long_sequence_gb300 import build as cuda_build
from tests.test_dense_convergence_host import FENCES
from tests.wide_turns import BITS, turns

OK, INVALID, UNSUPPORTED, OVERFLOW, WORKSPACE = 0, 1, 2, 3, 7
vp, i32, i64, f32, f64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                              ctypes.c_size_t)
A = [0x10000000 * (k + 1) for k in range(14)]      # addresses that nothing reads
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_long_sequence_gb300", "csrc")


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(cuda_build.build())
    sig = {
        "diffuser_rope_frequencies": [i32, f64, i32, f64, f64, vp, vp],
        "diffuser_rope": [vp, vp, i32, i64, i64, i64, i64, i32, vp, i32, i32, f32, vp, i64, vp, vp, vp],
        "diffuser_rope_backward": [vp, vp, i32, i64, i64, i64, i64, i32, vp, i32, i32, f32, vp, i64, vp, vp, vp],
        "diffuser_block_means": [vp, i64, i64, i64, i32, vp, i64, vp, vp],
        "diffuser_select_blocks": [vp, vp, i64, i64, i64, i64, i64, i32, i32, i32, i32, i32, vp, vp, vp, vp],
        "diffuser_selected_attention_workspace_size": [i64, i64, i64, i64, i64, i32, i32, vp],
        "diffuser_selected_attention": [vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp],
        "diffuser_selected_attention_backward_workspace_size": [i64, i64, i64, i64, i64, i32, i32, vp],
        "diffuser_selected_attention_backward": [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, i32, i32, vp, vp,
                                                 vp, vp, vp, vp, sz, vp],
    }
    for name, args in sig.items():
        getattr(lib, name).argtypes = args
    return lib


# ---------------------------------------------------------------- frequencies
@pytest.mark.parametrize("change,status", [
    (dict(scaling=-1), UNSUPPORTED), (dict(scaling=4), UNSUPPORTED), (dict(theta=0.5), INVALID),
    (dict(theta=float("nan")), INVALID), (dict(theta=float("inf")), INVALID), (dict(rot=0), INVALID), (dict(rot=-16), INVALID),
    (dict(rot=80), INVALID), (dict(rot=24), UNSUPPORTED), (dict(factor=0.5), INVALID), (dict(factor=float("nan")), INVALID),
    (dict(factor=float("inf")), INVALID), (dict(scaling=3, L=0.0), INVALID), (dict(scaling=3, L=float("nan")), INVALID),
    (dict(scaling=2, theta=1e300, factor=1e30), INVALID), (dict(out=None), INVALID), (dict(mag=None), INVALID)])
def test_frequency_refusals(lib, change, status):
    out, mag = (f64 * 32)(), f64()
    c = dict(dict(scaling=1, theta=1e4, rot=64, factor=4.0, L=4096.0, out=ctypes.addressof(out), mag=ctypes.addressof(mag)),
             **change)
    assert lib.diffuser_rope_frequencies(*c.values()) == status


def test_frequencies_without_a_scaling_read_no_factor(lib):
    out, mag = (f64 * 32)(), f64()
    assert lib.diffuser_rope_frequencies(0, 1e4, 64, float("nan"), float("nan"), ctypes.addressof(out), ctypes.addressof(mag)) == OK
    assert out[0] == 1.0 and mag.value == 1.0


MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "turns.h"
int main(int argc, char** argv) {
    for (int k = 1; k < argc; ++k) {
        uint64_t hi, lo;
        const double f = std::strtod(argv[k], nullptr);
        dfs::turns::fill_given(&hi, &lo, &f, 1);
        std::printf("%llx %llx\n", (unsigned long long)hi, (unsigned long long)lo);
    }
}
"""


def test_turns_of_given_frequencies(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    given = [0.0, 1.0, 4.0, 0.1, 1e-4, 1e-30, 1e-300, 5e-324, 3.9999999999999996, 2.718281828459045, 1.0 / 3.0]
    src, exe = tmp_path / "given.cpp", tmp_path / "given"
    src.write_text(MAIN)
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe), *(f.hex() for f in given)], check=True, capture_output=True, text=True).stdout
    per_turn = Fraction(turns(1.0, 16)[0], 1 << BITS)            # 1 / (2 pi)
    for f, line in zip(given, out.splitlines()):
        hi, lo = (int(x, 16) for x in line.split())
        want = Fraction(f) * per_turn
        # the constant and the product are each rounded down by less than 2^-126 of themselves, and the last place is cut
        assert abs(Fraction((hi << 64) | lo, 1 << 128) - want) <= want / (1 << 125) + Fraction(1, 1 << 128), f


# ---------------------------------------------------------------- rotation
FREQ = (f64 * 32)(*[1.0] * 32)
ROPE = dict(Q=A[0], K=A[1], dtype=1, B=1, Hq=2, Hk=2, n=4, d=64, freq=ctypes.addressof(FREQ), rot=64, inter=0, mag=1.0,
            pos=None, off=0, Qo=A[2], Ko=A[3])


def frequencies(x):
    arr = (f64 * 32)(*[1.0] * 32)
    arr[31] = x
    return arr


@pytest.mark.parametrize("name", ["diffuser_rope", "diffuser_rope_backward"])
@pytest.mark.parametrize("change,status", [
    (dict(d=128), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=80), INVALID),
    (dict(rot=0), INVALID), (dict(rot=-16), INVALID), (dict(freq=None), INVALID), (dict(freq=-0.1), INVALID),
    (dict(freq=4.1), INVALID), (dict(freq=float("nan")), INVALID), (dict(mag=0.0), INVALID), (dict(mag=float("nan")), INVALID),
    (dict(mag=float("inf")), INVALID), (dict(B=-1), INVALID), (dict(n=-1), INVALID), (dict(Hq=0), INVALID),
    (dict(Hk=5000), INVALID), (dict(B=1 << 31), INVALID), (dict(B=1 << 30, n=1 << 30), OVERFLOW), (dict(Q=None), INVALID),
    (dict(K=None), INVALID), (dict(Qo=None), INVALID), (dict(Ko=A[3] + 2), INVALID), (dict(pos=A[4] + 4), INVALID),
    (dict(Qo=A[0] + 16), INVALID), (dict(Qo=A[1]), INVALID), (dict(Ko=A[2]), INVALID), (dict(pos=A[2]), INVALID)])
def test_rope_refusals(lib, name, change, status):
    keep = None
    if isinstance(change.get("freq"), float):
        keep = frequencies(change["freq"])
        change = dict(freq=ctypes.addressof(keep))
    c = dict(ROPE, **change)
    assert getattr(lib, name)(*[c[k] for k in ROPE], None) == status


def test_rope_of_no_tokens(lib):
    for change in (dict(n=0), dict(B=0)):
        c = dict(ROPE, Q=None, K=None, Qo=None, Ko=None, **change)
        assert lib.diffuser_rope(*[c[k] for k in ROPE], None) == OK


# ---------------------------------------------------------------- means, choice, attention
MEANS = dict(K=A[0], B=2, Hk=2, m=100, d=64, lengths=None, recent=0, means=A[1])
SIZES = [(dict(d=128), UNSUPPORTED), (dict(m=(1 << 20) + 1), UNSUPPORTED), (dict(B=-1), INVALID), (dict(m=-1), INVALID),
         (dict(Hk=0), INVALID), (dict(B=1 << 31), INVALID), (dict(B=1 << 30, m=1 << 20), OVERFLOW),
         (dict(lengths=A[9] + 2), INVALID)]


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(recent=-1), INVALID), (dict(K=None), INVALID), (dict(means=None), INVALID), (dict(K=A[0] + 8), INVALID),
    (dict(means=A[0]), INVALID), (dict(lengths=A[1]), INVALID), (dict(Hk=5000), INVALID)])
def test_means_refusals(lib, change, status):
    c = dict(MEANS, **change)
    assert lib.diffuser_block_means(*[c[k] for k in MEANS], None) == status


SELECT = dict(Q=A[0], means=A[1], B=2, Hq=4, Hk=2, n=10, m=1000, d=64, top=8, sink=1, local=2, causal=1, lengths=None,
              starts=None, blocks=A[2])
QUERIES = [(dict(Hq=5), INVALID), (dict(Hq=8192, Hk=2), INVALID), (dict(n=-1), INVALID), (dict(top=0), UNSUPPORTED),
           (dict(top=65), UNSUPPORTED), (dict(n=(1 << 20) + 1), UNSUPPORTED),
           (dict(B=1, Hq=4096, Hk=1, n=1 << 20, m=64, top=1), OVERFLOW), (dict(starts=A[9] + 1), INVALID), (dict(Q=None), INVALID),
           (dict(Q=A[0] + 2), INVALID), (dict(blocks=A[2] + 4), INVALID), (dict(blocks=None), INVALID)]


@pytest.mark.parametrize("change,status", SIZES + QUERIES + [
    (dict(sink=-1), INVALID), (dict(local=-1), INVALID), (dict(sink=7, local=2), INVALID), (dict(sink=5, causal=0), OK),
    (dict(sink=6, causal=0), INVALID), (dict(local=1 << 30, causal=0), INVALID), (dict(means=None), INVALID),
    (dict(blocks=A[0]), INVALID), (dict(blocks=A[1]), INVALID), (dict(starts=A[2]), INVALID)])
def test_select_refusals(lib, change, status):
    c = dict(SELECT, **change)
    if status == OK:                                          # accepted sizes, nothing to do
        c.update(n=0, Q=None, blocks=None)
    assert lib.diffuser_select_blocks(*[c[k] for k in SELECT], None) == status


ATTEND = dict(Q=A[0], K=A[1], V=A[2], blocks=A[3], B=2, Hq=4, Hk=2, n=10, m=1000, d=64, top=8, causal=1, lengths=None,
              starts=None, out=A[4], lse=A[5], ws=None, bytes=0)


@pytest.mark.parametrize("change,status", SIZES + QUERIES + [
    (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(V=A[2] + 8), INVALID), (dict(out=None), INVALID),
    (dict(out=A[0]), INVALID), (dict(out=A[4] + 8), INVALID), (dict(lse=A[5] + 4), INVALID), (dict(lse=A[4]), INVALID),
    (dict(lse=A[3]), INVALID), (dict(lengths=A[4]), INVALID), (dict(n=1000), WORKSPACE), (dict(n=1000, ws=A[6], bytes=100), WORKSPACE),
    (dict(n=1000, ws=A[6] + 16, bytes=1 << 30), WORKSPACE), (dict(n=1000, ws=A[1], bytes=1 << 27), INVALID)])
def test_attention_refusals(lib, change, status):
    c = dict(ATTEND, **change)
    assert lib.diffuser_selected_attention(*[c[k] for k in ATTEND], None) == status


BACK = dict(Q=A[0], K=A[1], V=A[2], blocks=A[3], out=A[4], lse=A[5], dOut=A[6], B=2, Hq=4, Hk=2, n=10, m=1000, d=64, top=8,
            causal=1, lengths=None, starts=None, dQ=A[7], dK=A[8], dV=A[9], ws=A[10], bytes=1 << 27)


@pytest.mark.parametrize("change,status", [x for x in SIZES if "lengths" not in x[0]] + [x for x in QUERIES if "starts" not in x[0]] + [
    (dict(K=None), INVALID), (dict(out=None), INVALID), (dict(lse=None), INVALID), (dict(dOut=None), INVALID),
    (dict(dQ=None), INVALID), (dict(dK=None), INVALID), (dict(dV=A[9] + 2), INVALID), (dict(dQ=A[6]), INVALID),
    (dict(dK=A[1]), INVALID), (dict(dV=A[8]), INVALID), (dict(lengths=A[12] + 2), INVALID), (dict(starts=A[12] + 2), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=A[10] + 64), WORKSPACE), (dict(bytes=1000), WORKSPACE), (dict(ws=A[4]), INVALID)])
def test_backward_refusals(lib, change, status):
    c = dict(BACK, **change)
    assert lib.diffuser_selected_attention_backward(*[c[k] for k in BACK], None) == status


def test_workspace_sizes(lib):
    b = sz()
    for name in ("diffuser_selected_attention_workspace_size", "diffuser_selected_attention_backward_workspace_size"):
        size = getattr(lib, name)
        assert size(1, 2, 1, 10, 100, 64, 4, None) == INVALID and size(1, 2, 1, 10, 100, 32, 4, ctypes.addressof(b)) == UNSUPPORTED
        for empty in ((0, 2, 1, 10, 100), (1, 2, 1, 0, 100), (1, 2, 1, 10, 0)):
            assert size(*empty, 64, 4, ctypes.addressof(b)) == OK and b.value == 0
        assert size(1, 16, 16, 16384, 16384, 64, 16, ctypes.addressof(b)) == OK and (1 << 30) < b.value < (3 << 30)
        # a group of units at a time: eight times the queries need less than twice the partial sums' place
        at = b.value
        assert size(8, 16, 16, 16384, 16384, 64, 16, ctypes.addressof(b)) == OK and b.value < 2.5 * at
    assert lib.diffuser_selected_attention_workspace_size(16, 16, 4, 1, 65536, 64, 16, ctypes.addressof(b)) == OK and b.value == 0


# ---------------------------------------------------------------- warp-wide instructions
CALLS = r"ptx::(?:named_barrier_sync|tmem_ld\w*_issue|tmem_ld\d+|tmem_st\w+|tmem_alloc|tmem_dealloc)\s*\("
BEFORE = r"__syncwarp\(\);\s*(?:if \(warp == 0\) )?" + FENCES


def apart(text):
    """Warp-wide tensor memory and barrier instructions that do not follow a __syncwarp(), directly or behind
    another load: line numbers."""
    code = re.sub(r"//[^\n]*", "", text)
    return [code.count("\n", 0, m.start()) + 1 for m in re.finditer(CALLS, code)
            if not re.search(BEFORE + r"(?:ptx::tmem_ld32_issue\([^;]*;\s*)*$", code[:m.start()])]


@pytest.mark.parametrize("path", [os.path.join(CSRC, f) for f in ("select_tiles.cu", "selected_attention.cu", "selected_backward.cu")],
                         ids=os.path.basename)
def test_lanes_meet_before_warp_wide_instructions(path):
    with open(path) as f:
        text = f.read()
    assert apart(text) == []
    assert len(re.findall(CALLS, text)) >= 3
    assert apart("if (lead) go();\nptx::named_barrier_sync(1, 64);") == [2]
