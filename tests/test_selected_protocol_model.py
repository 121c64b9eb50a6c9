"""A host model of the barriers of the attention over chosen key blocks.

`selected_tiles_kernel` (csrc/selected_attention.cu) and `selected_grads_kernel`
(csrc/selected_backward.cu) walk over tiles with all warps alike: block-wide
barriers between the hand-overs, and mbarriers that the tensor core's commits
complete.  The sequences are restated here, the tensor core as a role of its own
that takes its products in order, and played out (tests/barrier_model.py): every
role must finish for any number of tiles, and no wait may find its mbarrier two
phases ahead.  A second model follows what each buffer holds: a copy or a store
into a buffer while a product or a copy engine may still read it is an overrun.
It checks the protocol as designed; keeping it in step with the kernels is a
review duty whenever either changes.
"""
import pytest

from tests.barrier_model import play

WARPS = 4


def W(bar, k):
    return ("w", bar, k)


def A(bar):
    return ("a", bar)


def meet(name, k):
    """A block-wide barrier: arrive, then wait for the others."""
    return [A(name), W(name, k)]


def forward(tiles, missing=None):
    """Roles of the forward: warps, and the tensor core fed by warp 0."""
    counts = {"top": WARPS, "mid": WARPS, "s": 1, "o": 1, "ask_s": 1, "ask_o": 1}
    warps = []
    for w in range(WARPS):
        ops = []
        for x in range(tiles):
            ops += meet("top", x)
            if w == 0:
                ops.append(A("ask_s"))
            ops.append(W("s", x))
            if not (missing == "warp" and w == 2 and x == 1):
                ops += meet("mid", x)
            if w == 0:
                ops.append(A("ask_o"))
            ops.append(W("o", x))
        warps.append(ops)
    core = [op for x in range(tiles) for op in (W("ask_s", x), A("s"), W("ask_o", x), A("o"))]
    if missing == "commit" and tiles:
        core.pop()
    return play(warps + [core], counts)


@pytest.mark.parametrize("tiles", range(1, 9))
def test_forward_completes(tiles):
    assert forward(tiles) == "done"


def test_planted_mistakes_of_the_forward():
    assert forward(4, "commit") == "stalled"                 # the last product's commit left out
    assert forward(4, "warp") == "stalled"                   # a warp that passes a barrier by


def backward(tiles):
    """Three mbarriers: S and dout V^T, dq, and dv with dk; dq leaves by P's place, behind a bulk copy's read."""
    counts = {"top": WARPS, "free": WARPS, "mid": WARPS, "s": 1, "q": 1, "kv": 1, "ask_s": 1, "ask_q": 1}
    warps = []
    for w in range(WARPS):
        ops = []
        for x in range(tiles):
            ops += meet("top", x)
            if w == 0:
                ops.append(A("ask_s"))
            ops.append(W("s", x))
            ops += meet("free", x)
            ops += meet("mid", x)
            if w == 0:
                ops.append(A("ask_q"))
            ops += [W("q", x), W("kv", x)]
        warps.append(ops)
    core = [op for x in range(tiles) for op in (W("ask_s", x), A("s"), W("ask_q", x), A("q"), A("kv"))]
    return play(warps + [core], counts)


@pytest.mark.parametrize("tiles", range(1, 9))
def test_backward_completes(tiles):
    assert backward(tiles) == "done"


# ---------------------------------------------------------------- what the buffers hold
def hazards_forward(blocks, wait_for_s=True):
    """One block of threads' order of events over tiles of the given key blocks: (buffer, content) that
    each product reads against what is there, copies being there as soon as they are issued (the worst)."""
    held, bad = {}, []
    side = 0

    def load(buf, what):
        held[buf] = what
    load("keys", blocks[0]), load(("values", 0), blocks[0]), load("queries", 0)
    for x, block in enumerate(blocks):
        def s_product():
            bad.extend((x, b) for b, what in (("keys", block), ("queries", x)) if held[b] != what)
        if wait_for_s:
            s_product()
        here = side
        if x + 1 < len(blocks):              # issued once S is there
            if blocks[x + 1] != block:
                side ^= 1
                load("keys", blocks[x + 1]), load(("values", side), blocks[x + 1])
            load("queries", x + 1)
        if not wait_for_s:
            s_product()
        bad.extend((x, "values") for _ in (0,) if held[("values", here)] != block)      # O = P V, later
    return bad


RUNS = [[0], [0, 0], [0, 1], [0, 1, 2, 3], [0, 0, 1, 1, 1, 2], [3, 4, 4, 5, 6, 6, 6]]


@pytest.mark.parametrize("blocks", RUNS)
def test_forward_buffers(blocks):
    assert hazards_forward(blocks) == []


def test_forward_buffers_without_the_wait():
    assert hazards_forward([0, 1, 2], wait_for_s=False) != []


def hazards_backward(blocks, early=False):
    """Likewise: two stages of dout and queries; keys and values follow once dq is there."""
    held, bad = {}, []
    held["block"], held[0] = blocks[0], 0
    for x, block in enumerate(blocks):
        bad.extend((x, "S") for _ in (0,) if held["block"] != block or held[x & 1] != x)
        if x + 1 < len(blocks):
            held[(x + 1) & 1] = x + 1        # its last reader, dv and dk of x - 1, has been waited for
            if early and blocks[x + 1] != block:
                held["block"] = blocks[x + 1]
        bad.extend((x, "dq") for _ in (0,) if held["block"] != block)
        bad.extend((x, "dv, dk") for _ in (0,) if held[x & 1] != x)
        if x + 1 < len(blocks) and blocks[x + 1] != block:
            held["block"] = blocks[x + 1]    # dq is there
    return bad


@pytest.mark.parametrize("blocks", RUNS)
def test_backward_buffers(blocks):
    assert hazards_backward(blocks) == []


def test_backward_buffers_copied_too_early():
    assert hazards_backward([0, 1, 2], early=True) != []


# ---------------------------------------------------------------- shares of tiles
def share_begin(tiles, share, shares):
    return tiles * share // shares


def share_of_tile(tiles, t, shares):
    return ((t + 1) * shares - 1) // tiles


@pytest.mark.parametrize("shares", [1, 2, 3, 7, 28, 608])
def test_shares(shares):
    """Every tile has one share, every share of a unit has tiles, and the parts of a block that the shares
    leave are those that the joining kernel adds up."""
    for tiles in list(range(1, 40)) + [607, 608, 609, 5000]:
        n = min(shares, tiles)
        runs = [range(share_begin(tiles, j, n), share_begin(tiles, j + 1, n)) for j in range(n)]
        assert all(len(r) > 0 for r in runs) and [t for r in runs for t in r] == list(range(tiles))
        assert all(share_of_tile(tiles, t, n) == j for j, r in enumerate(runs) for t in r)
        for begin, end in ((0, tiles), (0, 1), (tiles // 3, tiles // 3 + 1 + tiles // 4)):
            if not begin < end <= tiles:
                continue
            left = set()
            for j, r in enumerate(runs):
                if r.start < end and begin < r.stop and not (begin >= r.start and end <= r.stop):
                    left.add((j, 0 if begin < r.start else 1))
            first, last = share_of_tile(tiles, begin, n), share_of_tile(tiles, end - 1, n)
            joined = set() if first == last else {(first + x, 1 if x == 0 else 0) for x in range(last - first + 1)}
            assert left == joined
