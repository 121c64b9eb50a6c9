"""Host models of the mbarrier protocols of csrc/dense_pair.cu's other two kernels, played out by
tests/barrier_model.py: K split over the pairs of a cluster (dense_pair_split_kernel), and both
gradients in one launch (dense_grads_kernel).  They check the protocols as designed; keeping them
in step with the kernels is a review duty whenever either changes.

Both: a pair's full barriers are those of its first CTA and take one arrival (the expected bytes)
and both CTAs' copies; a commit arrives on both CTAs' empty barriers.  Split: pair s of the
cluster uses the barriers of the CTAs of rank 2 s and 2 s + 1, each CTA drains its own, and the
cluster barriers wait for every role of every CTA.  Gradients: 8 epilogue warps a CTA, a tile's K
steps depend on its product, an accumulator is released after its last store, and before the first
one the epilogue warps of a CTA sum the bias gradient between named barriers of their own.
"""
import random

import pytest

from tests.barrier_model import play


def wait(bar, k):
    return ("w", bar, k)


def arrive(bar):
    return ("a", bar)


def loader(tag, rank, steps, stages, drain=True):
    ops = []
    for n in range(steps):
        s = n % stages
        if n >= stages:
            ops.append(wait(("empty", tag, rank, s), n // stages - 1))
        ops.append(arrive(("full", tag, s)))
    for s in range(stages):
        uses = (steps - s + stages - 1) // stages
        if uses > 0 and drain:
            ops.append(wait(("empty", tag, rank, s), uses - 1))
    return ops


def step(tag, n, stages, both=True):
    s = n % stages
    return [wait(("full", tag, s), n // stages)] + [arrive(("empty", tag, r, s)) for r in range(2 if both else 1)]


def ring(tag, stages):
    counts = {("full", tag, s): 2 for s in range(stages)}
    counts.update({("empty", tag, r, s): 1 for r in range(2) for s in range(stages)})
    return counts


def split(k_blocks, splits, stages, commit_both=True, accs=1):
    counts, roles = {}, []
    for p in range(splits):
        steps = k_blocks * (p + 1) // splits - k_blocks * p // splits
        assert steps >= 1                                     # the launcher halves the split otherwise
        counts.update(ring(p, stages))
        counts.update({("acc", p, r): accs for r in range(2)})
        for r in range(2):
            roles.append(loader(p, r, steps, stages))
            roles.append([])                                  # warp 1
            if r == 0:
                for n in range(steps):
                    roles[-1] += step(p, n, stages, commit_both)
                roles[-1] += [arrive(("acc", p, 0)), arrive(("acc", p, 1))]
            roles += [[wait(("acc", p, r), 0)] for _ in range(8)]     # each lays its part into the ring
    # the barrier before the sums, and the one before anybody leaves
    counts["cluster"] = len(roles)
    for k in range(2):
        for ops in roles:
            ops += [arrive("cluster"), wait("cluster", k)]
    return play(roles, counts)


@pytest.mark.parametrize("stages", [5, 6])
@pytest.mark.parametrize("splits", [2, 4])
def test_split_pairs_complete(splits, stages):
    for k_blocks in (splits, splits + 1, 7, 13, 24, 61):
        assert split(k_blocks, splits, stages) == "done"


def test_split_model_detects_planted_mistakes():
    assert split(40, 2, 5, commit_both=False) == "stalled"    # the second CTA's stages never come free
    assert split(40, 2, 5, accs=2) == "stalled"


WARPS = 8


def grads(tiles, stages, bias_rounds=0, releases=2 * WARPS, named=WARPS, buffers=2):
    """tiles: K steps of a pair's tiles in turn (the longer product's first)."""
    counts = ring(0, stages)
    counts.update({("accF", r, b): 1 for r in range(2) for b in range(2)})
    counts.update({("accE", b): releases for b in range(2)})
    counts.update({("named", r): named for r in range(2)})
    total = sum(tiles)
    roles = [loader(0, r, total, stages) for r in range(2)]
    mma, n = [], 0
    for lt, steps in enumerate(tiles):
        if lt >= buffers:
            mma.append(wait(("accE", lt & 1), lt // 2 - 1))
        for _ in range(steps):
            mma += step(0, n, stages)
            n += 1
        mma += [arrive(("accF", 0, lt & 1)), arrive(("accF", 1, lt & 1))]
    roles.append(mma)
    for r in range(2):
        for _ in range(WARPS):
            ops = []
            for k in range(2 * bias_rounds):
                ops += [arrive(("named", r)), wait(("named", r), k)]
            for lt in range(len(tiles)):
                ops += [wait(("accF", r, lt & 1), lt // 2), arrive(("accE", lt & 1))]
            roles.append(ops)
    return play(roles, counts)


@pytest.mark.parametrize("stages", [5, 6])
@pytest.mark.parametrize("bias_rounds", [0, 1, 3])
def test_gradients_complete(stages, bias_rounds):
    rng = random.Random(stages)
    cases = [[], [1], [9, 2], [64] * 2 + [12] * 5, [3, 1, 1, 1, 1]]
    cases += [[rng.randint(1, 20)] * rng.randint(1, 4) + [rng.randint(1, 6)] * rng.randint(0, 7) for _ in range(12)]
    for tiles in cases:
        assert grads(tiles, stages, bias_rounds) == "done"


def test_gradients_model_detects_planted_mistakes():
    assert grads([4, 4, 2, 2], 5, releases=2 * WARPS + 1) == "stalled"
    assert grads([4, 4], 5, bias_rounds=1, named=WARPS + 1) == "stalled"
    assert grads([1] * 6, 6, buffers=6) == "overrun"          # accumulators reused without a wait
