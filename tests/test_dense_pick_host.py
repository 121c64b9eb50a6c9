"""The rule that picks a dense product's kernel (csrc/dense_pick.cu), compiled for the host with
recorders in the launches' place: which kernel it takes at the sizes of tests/dense_sizes.py, for
every number of clusters that a device may hold, and that those sizes leave out no kernel."""
import os
import re
import shutil
import subprocess

import pytest

from tests import dense_sizes as sizes
from tests.test_dense_protocol_model import deal

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_long_sequence_gb300", "csrc")
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")
MAIN = r"""
#include <cstdio>
#include "dense_pick.cu"
namespace dfs {
int clusters[3];
long long steps128, steps256;
int dense_pair_clusters(int splits) { return clusters[splits >> 1]; }
int launch_dense_few(const DenseArgs&, cudaStream_t) { return std::printf(" few 0 0"), 0; }
int launch_dense_pair(DenseForm, const DenseArgs&, int bn, int splits, cudaStream_t) {
    return std::printf(" pair %d %d", bn, splits), 0;
}
int launch_dense_grads(const DenseArgs&, const DenseArgs&, const BiasSums&, int bn, cudaStream_t) {
    return std::printf(" grads %d", bn), 0;
}
int64_t dense_grads_steps(const DenseArgs&, int bn) { return bn == 256 ? steps256 : steps128; }
int launch_colsum(const BiasSums&, cudaStream_t) { return 0; }
}  // namespace dfs
int main() {
    using namespace dfs;
    int form, D, cols, gated;
    long long T;
    while (std::scanf("%d %lld %d %d %d %d %d %d %lld %lld", &form, &T, &D, &cols, &gated, &clusters[0], &clusters[1],
                      &clusters[2], &steps128, &steps256) == 10) {
        DenseArgs a{};
        a.rows = T;
        a.inner = D;
        a.cols = cols;
        a.gated = gated != 0;
        if (form == 3) launch_gradients(a, a, BiasSums{}, nullptr);
        else launch_dense((DenseForm)form, a, nullptr);
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def pick(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    d = tmp_path_factory.mktemp("pick")
    src, exe = d / "pick.cpp", d / "pick"
    src.write_text(MAIN)
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, "-I", os.path.join(CUDA, "include"), str(src), "-o", str(exe)], check=True)

    def run(calls):
        text = "\n".join(" ".join(str(int(x)) for x in c) for c in calls)
        out = subprocess.run([str(exe)], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(int(w) if w.isdigit() else w for w in line.split()) for line in out.splitlines()]
    return run


@pytest.mark.parametrize("name", sizes.FORMS)
def test_every_kernel_has_its_sizes(pick, name):
    form, gated, table = sizes.FORMS[name]
    want, calls = [], []
    for kernel, shapes in table.items():
        for T, D, F in shapes:
            for c in sizes.CLUSTERS:
                want.append(((T, D, F), c, kernel))
                calls.append((form, T, D, 2 * F if gated else F, gated, *c, 0, 0))
    got = pick(calls)
    assert len(got) == len(want)
    assert [(w[0], w[1], g) for w, g in zip(want, got)] == want


@pytest.mark.parametrize("name", sizes.FORMS)
def test_no_other_kernel_is_picked(pick, name):
    # over a grid of sizes the rule takes the table's kernels, and each of them somewhere
    form, gated, table = sizes.FORMS[name]
    grid = [8, 33, 64, 65, 136, 300, 520, 777, 1032, 1544, 2816, 4096, 8200, 30000]
    calls = [(form, T, -(-D // 8) * 8, -(-F // 8) * 8 * (2 if gated else 1), gated, 76, 34, 15, 0, 0)
             for T in grid for D in grid for F in grid]
    assert set(pick(calls)) == set(table)


def grads_steps(T, D, cols, bn, pairs):
    """The busiest pair's K steps of both gradients in one launch (csrc/dense_pair.cu's dealing)."""
    up = lambda x, y: -(-x // y)
    x = up(T, 256) * up(D, bn), up(cols, 64)                    # dX [T][D] over cols
    w = up(cols, 256) * up(D, bn), up(T, 64)                    # dW [cols][D] over T
    (longs, long_steps), (shorts, short_steps) = (w, x) if w[1] >= x[1] else (x, w)
    return max(len(a) * long_steps + len(b) * short_steps for a, b in deal(longs, long_steps, shorts, short_steps, pairs))


def test_both_gradients(pick):
    want, calls = [], []
    for kind, shapes in sizes.BOTH_GRADIENTS.items():
        for T, D, F in shapes:
            for c in sizes.CLUSTERS:
                want.append(kind)
                calls.append((3, T, D, F, 0, *c, *(grads_steps(T, D, F, bn, c[0]) for bn in (128, 256))))
    got = [g if g[0] == "grads" else (g[0], g[3]) for g in pick(calls)]
    assert list(zip(calls, got)) == list(zip(calls, want))


def test_the_instantiations_are_these():
    # the kernels that csrc/dense_pair.cu's launchers can reach are those of the tables
    with open(os.path.join(CSRC, "dense_pair.cu")) as f:
        text = f.read()
    body = text[text.index("int launch_dense_pair("):]
    found = {(a == "true", b == "true", g == "true", int(n))
             for a, b, g, n in re.findall(r"launch_as<(\w+), (\w+), (\w+), (\d+)>", body)}
    tables = {(False, False, False): sizes.FORWARD, (False, False, True): sizes.GATED, (False, True, False): sizes.INPUT_GRADIENT,
              (True, True, False): sizes.WEIGHT_GRADIENT}
    assert found == {(*k, n) for k, t in tables.items() for kind, n, _ in t if kind == "pair"}
    assert set(re.findall(r"launch_grads_as<(\d+)>", text)) == {str(n) for kind, n in sizes.BOTH_GRADIENTS if kind == "grads"}
