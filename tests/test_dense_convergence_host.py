"""Warp-wide (.aligned) instructions of the dense and gated products are undefined where a
warp's lanes arrive apart: after a loop that some lanes leave early, a branch of one lane, or a
barrier wait that each lane polls for itself.  So every cluster barrier, named barrier and
accumulator load in csrc/dense_* comes directly after a __syncwarp() (fences of the thread's own
may stand between), in the wrapper or at the call."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_long_sequence_gb300", "csrc")
# calls whose wrappers leave the meeting to the caller, and the instruction of the one that does not
CALLS = r"ptx::(?:named_barrier_sync|tmem_ld\w*_issue|tmem_ld\d+)\s*\("
INSTRUCTION = r'asm volatile\(\s*"barrier\.cluster\.arrive'
FENCES = r"(?:ptx::tc_fence_(?:before|after)\(\);\s*)*"


def apart(text):
    """Where a warp-wide instruction does not directly follow a __syncwarp(): line numbers."""
    code = re.sub(r"//[^\n]*", "", text)
    return [code.count("\n", 0, m.start()) + 1 for m in re.finditer(f"{CALLS}|{INSTRUCTION}", code)
            if not re.search(r"__syncwarp\(\);\s*" + FENCES + r"$", code[:m.start()])]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "dense_*")))


@pytest.mark.parametrize("path", sources(), ids=os.path.basename)
def test_lanes_meet_before_warp_wide_instructions(path):
    with open(path) as f:
        assert apart(f.read()) == []


def test_the_instructions_are_found():
    text = "".join(open(p).read() for p in sources())
    # the cluster barrier's wrapper, the bias sums' two barriers, the three kernels' accumulator loads
    assert len(re.findall(INSTRUCTION, text)) == 1 and text.count("ptx::named_barrier_sync(") == 2
    assert len(re.findall(r"ptx::tmem_ld", text)) >= 3
    assert not re.search(r'"(?:bar\.sync|barrier\.sync|tcgen05\.ld)', text)     # none past the wrappers


def test_planted_mistakes_are_found():
    assert apart("if (lead) go();\nptx::named_barrier_sync(1, 64);") == [2]
    assert apart("__syncwarp();\nptx::tc_fence_after();\nptx::tmem_ld32(a, v);") == []
    assert apart('__syncwarp();\nfor (;;) {\nptx::tmem_ld32_issue(a, v);\n}') == [3]
    assert apart('void f() {\n    asm volatile("barrier.cluster.arrive.release.aligned;");\n}') == [2]
