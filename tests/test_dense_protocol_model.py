"""Host models of the dense products' mbarrier protocols (csrc/dense_pair.cu and
csrc/dense_few.cu), played out by tests/barrier_model.py: every role must finish for any
tile and K-step count, and no wait may find its barrier two phases ahead.  They check the
protocols as designed; keeping them in step with the kernels is a review duty whenever
either changes.

The pair kernel: CTA 0's full barriers take one arrival (the expected bytes) and both CTAs'
copies; a commit arrives on both CTAs' barriers; the accumulators are freed by the pair's
epilogue warps (16 a CTA, 8 for the gradients); a warp's residual barriers take one arrival
per load.
"""
import pytest

from tests.barrier_model import play

BUFS, WARPS = 2, 16


def wait(bar, k):
    return ("w", bar, k)


def arrive(bar):
    return ("a", bar)


def pair(my, k_blocks, stages, blocks=2, residual=False, pre=False, acc_empty=2 * WARPS, ring=True,
         live=lambda rank, warp, lt: 2):
    counts = {("full", s): 2 for s in range(stages)}       # the expect and the peer's copies
    for r in range(2):
        counts.update({("empty", r, s): 1 for s in range(stages)})
        counts.update({("accF", r, b): 1 for b in range(2)})
        counts.update({("res", r, w, b): 1 for w in range(WARPS) for b in range(BUFS)})
    counts.update({("accE", b): acc_empty for b in range(2)})
    roles = []
    for r in range(2):
        tma, n = [], 0
        for _ in range(my * k_blocks):
            s = n % stages
            if n >= stages and ring:
                tma.append(wait(("empty", r, s), n // stages - 1))
            tma.append(arrive(("full", s)))
            n += 1
        for s in range(stages):
            uses = (n - s + stages - 1) // stages
            if uses > 0:
                tma.append(wait(("empty", r, s), uses - 1))
        roles.append(tma)
    mma, n = [], 0
    for lt in range(my):
        if lt >= 2:
            mma.append(wait(("accE", lt & 1), lt // 2 - 1))
        for _ in range(k_blocks):
            s = n % stages
            mma += [wait(("full", s), n // stages), arrive(("empty", 0, s)), arrive(("empty", 1, s))]
            n += 1
        mma += [arrive(("accF", 0, lt & 1)), arrive(("accF", 1, lt & 1))]
    roles.append(mma)
    for r in range(2):
        for w in range(WARPS):
            ops, u, loads, waits = [], 0, [0] * BUFS, [0] * BUFS
            for lt in range(my):
                now = min(blocks, live(r, w, lt))

                def load(b):
                    ops.append(arrive(("res", r, w, b)))
                    loads[b] += 1
                    assert loads[b] - waits[b] <= 1, "a residual lands in a buffer that holds one"
                if residual and not pre:
                    for k in range(now):
                        load((u + k) % BUFS)
                ops.append(wait(("accF", r, lt & 1), lt // 2))
                if not now:
                    ops.append(arrive(("accE", lt & 1)))
                for k in range(now):
                    if residual and pre:
                        load((u + 1) % BUFS)
                    if k + 1 == now:
                        ops.append(arrive(("accE", lt & 1)))
                    u += 1 if pre else 0
                    if residual:
                        b = u % BUFS
                        ops.append(wait(("res", r, w, b), waits[b]))
                        waits[b] += 1
                    u += 1
            roles.append(ops)
    return play(roles, counts)


@pytest.mark.parametrize("stages", [5, 6])
@pytest.mark.parametrize("k_blocks", [1, 2, 6, 12])
def test_pair_protocol_completes(stages, k_blocks):
    for my in (0, 1, 2, 5):
        for residual in (False, True):
            for pre in (False, True):
                for blocks in (1, 2):
                    assert pair(my, k_blocks, stages, blocks, residual, pre) == "done"


def test_pair_protocol_with_ragged_tiles():
    # warps with some or no block inside the result
    for pre in (False, True):
        assert pair(5, 3, 5, residual=True, pre=pre, live=lambda r, w, lt: (r + 2 * w + lt) % 3) == "done"


def test_pair_model_detects_planted_mistakes():
    assert pair(4, 12, 5, acc_empty=2 * WARPS + 1) == "stalled"
    assert pair(4, 12, 5, ring=False) == "overrun"


def split(steps, stages, drain=True):
    counts = {("full", s): 1 for s in range(stages)}
    counts.update({("empty", s): 1 for s in range(stages)})
    counts["acc"] = 1
    tma, mma = [], []
    for n in range(steps):
        s = n % stages
        if n >= stages:
            tma.append(wait(("empty", s), n // stages - 1))
        tma.append(arrive(("full", s)))
        mma += [wait(("full", s), n // stages), arrive(("empty", s))]
    mma.append(arrive("acc"))
    for s in range(stages):
        uses = (steps - s + stages - 1) // stages
        if uses > 0 and drain:
            mma.append(wait(("empty", s), uses - 1))
    return play([tma + [wait("acc", 0)], mma + [wait("acc", 0)], [wait("acc", 0)]], counts)


@pytest.mark.parametrize("stages", range(1, 9))
def test_split_protocol_completes(stages):
    for steps in range(1, 30):
        assert split(steps, stages) == "done"


def deal(longs, long_steps, shorts, short_steps, pairs):
    """csrc/dense_pair.cu's deal_tiles, long_tile and short_tile: the long and short tiles of each pair."""
    per, na = divmod(longs, pairs)
    nb = pairs - na
    load_b = per * long_steps
    load_a = load_b + long_steps
    b = -(-long_steps // short_steps)
    to_b = nb * b if na else 0
    if not na or to_b >= shorts:
        to_b = shorts
    else:
        rest = shorts - to_b
        to_b += rest // pairs * nb
        last = rest % pairs
        lower = load_b + b * short_steps <= load_a
        first = min(last, nb if lower else na)
        to_b += first if lower else last - first
    to_a = shorts - to_b
    bs, br = divmod(to_b, nb)
    as_, ar = divmod(to_a, na) if na else (0, 0)
    out = []
    for p in range(pairs):
        long = [k * pairs + p for k in range(per + (p < na))]
        if p < na:
            short = [k * na + p for k in range(as_ + (p < ar))]
        else:
            short = [na * as_ + ar + k * nb + p - na for k in range(bs + (p - na < br))]
        out.append((long, short))
    return out


@pytest.mark.parametrize("pairs", [1, 2, 7, 76])
def test_gradient_tiles_are_dealt_once_and_evenly(pairs):
    import random
    rng = random.Random(pairs)
    cases = [(64, 256, 256, 64), (88, 256, 256, 88), (9, 128, 96, 12), (1, 5, 0, 1), (pairs, 3, 2 * pairs, 3)]
    cases += [(rng.randint(1, 400), rng.randint(1, 300), rng.randint(0, 600), 1) for _ in range(200)]
    for longs, long_steps, shorts, short_steps in cases:
        short_steps = short_steps if short_steps > 1 else rng.randint(1, long_steps)
        n = min(pairs, longs + shorts)
        shares = deal(longs, long_steps, shorts, short_steps, n)
        assert sorted(t for long, _ in shares for t in long) == list(range(longs))      # every tile once
        assert sorted(t for _, short in shares for t in short) == list(range(shorts))
        most = max(len(long) * long_steps + len(short) * short_steps for long, short in shares)
        loads = [0] * n                                  # the same by the greedy rule
        for steps, count in ((long_steps, longs), (short_steps, shorts)):
            for _ in range(count):
                k = loads.index(min(loads))
                loads[k] += steps
        assert most <= max(loads) + short_steps
