"""The rotation alone, the means of key blocks, the choice of blocks and the attention over them,
against their definitions in 64 bits.

Bounds count roundings: half a step of a type, u = finfo.eps / 2 of the value (bf16 2^-8, fp32 2^-24)."""
import math

import pytest
import torch

from tests import selected_reference as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def dl():
    from sparse_long_sequence_gb300 import binding
    return binding


def normal(gen, *shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32)


def cuda(x):
    return None if x is None else x.cuda()


# ---------------------------------------------------------------- rotation
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,Hq,Hk,n,rot,inter,scaling,pos", [
    (1, 1, 1, 1, 64, False, "NONE", None), (2, 3, 1, 5, 64, False, "YARN", "far"), (3, 12, 4, 77, 32, True, "NTK", "far"),
    (1, 2, 2, 130, 16, False, "LINEAR", None), (2, 1, 5, 33, 48, True, "YARN", "negative")])
def test_rope(dl, dtype, B, Hq, Hk, n, rot, inter, scaling, pos):
    gen = torch.Generator().manual_seed(1)
    q, k = normal(gen, B, Hq, n, 64, dtype=dtype), normal(gen, B, Hk, n, 64, dtype=dtype)
    at = torch.arange(n).expand(B, -1).clone()
    if pos == "far":
        at = at + torch.randint(0, 1 << 20, (B, 1), generator=gen)
    if pos == "negative":
        at = -at
    freq, mag = dl.diffuser_rope_frequencies(rot, 10000.0, getattr(dl, "DIFFUSER_ROPE_" + scaling), 4.0, 4096)
    given = None if pos is None else at.cuda()
    back = dl.diffuser_rope_backward
    for call, sign in ((dl.diffuser_rope, 1), (back, -1)):
        out = call(q.cuda(), k.cuda(), freq, magnitude=mag, interleaved=inter, positions=given)
        for x, y in zip((q, k), out):
            want = ref.rope(x, freq, mag, inter, sign * at)
            # a cosine's argument is off by 2^-31 turns and its value by 2^-23; three fp32 operations
            pair = 2.0 ** -21 * mag * x.double().abs().amax(-1, keepdim=True) * 2
            err = (y.double().cpu() - want).abs()
            assert (err <= U[dtype] * want.abs() + pair).all(), err.max()
        # in place, and an offset in place of the positions
        a, b = q.cuda(), k.cuda()
        given_back = call(a, b, freq, magnitude=mag, interleaved=inter, positions=given, **dict(zip(
            ("Qo", "Ko") if sign > 0 else ("dQ", "dK"), (a, b))))
        assert given_back[0] is a and torch.equal(a, out[0]) and torch.equal(b, out[1])


def test_rope_gradient_is_the_transpose(dl):
    gen = torch.Generator().manual_seed(2)
    q, k, dq, dk = (normal(gen, 2, 3, 40, 64, dtype=F32).cuda() for _ in range(4))
    freq, mag = dl.diffuser_rope_frequencies(32, 10000.0, dl.DIFFUSER_ROPE_YARN, 8.0, 2048)
    yq, yk = dl.diffuser_rope(q, k, freq, magnitude=mag, position_offset=1000)
    gq, gk = dl.diffuser_rope_backward(dq, dk, freq, magnitude=mag, position_offset=1000)
    for y, d, x, g in ((yq, dq, q, gq), (yk, dk, k, gk)):
        a, b = (y.double() * d.double()).sum(), (x.double() * g.double()).sum()
        # 2 x 7680 products of values with a relative error of a few 2^-23
        assert abs(a - b) <= 2.0 ** -21 * (y.double() * d.double()).abs().sum()


def test_rope_frequencies(dl):
    r, s, L = 48, 4.0, 4096.0
    base, one = dl.diffuser_rope_frequencies(r)
    assert one == 1.0 and [base[i] for i in range(24)] == pytest.approx([10000.0 ** (-2 * i / r) for i in range(24)], rel=1e-14)
    lin, _ = dl.diffuser_rope_frequencies(r, 10000.0, dl.DIFFUSER_ROPE_LINEAR, s)
    assert list(lin) == pytest.approx([f / s for f in base], rel=1e-14)
    ntk, _ = dl.diffuser_rope_frequencies(r, 10000.0, dl.DIFFUSER_ROPE_NTK, s)
    assert ntk[0] == 1.0 and ntk[23] == pytest.approx(base[23] / s, rel=1e-12)    # the slowest is stretched in full
    yarn, mag = dl.diffuser_rope_frequencies(r, 10000.0, dl.DIFFUSER_ROPE_YARN, s, L)
    assert mag == pytest.approx(1 + 0.1 * math.log(s), rel=1e-14)
    for f, y in zip(base, yarn):
        turns = L * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        assert y == pytest.approx(f * (keep + (1 - keep) / s), rel=1e-13)


# ---------------------------------------------------------------- means of key blocks
@pytest.mark.parametrize("B,Hk,m,lengths,recent", [
    (1, 1, 1, None, 0), (2, 3, 64, None, 0), (2, 2, 65, None, 0), (1, 2, 1000, None, 0), (3, 2, 300, [0, 64, 300], 0),
    (4, 1, 300, [1, 65, 128, 129], 1), (2, 2, 300, [200, 300], 130), (2, 1, 130, [-5, 999], 1), (1, 1, 200, [200], 5000)])
def test_block_means(dl, B, Hk, m, lengths, recent):
    gen = torch.Generator().manual_seed(3)
    K = normal(gen, B, Hk, m, 64)
    for b, x in enumerate(lengths or []):
        K[b, :, max(0, min(m, x)):] = math.nan               # not read
    old = normal(gen, B, Hk, -(-m // 64), 64)
    got = dl.diffuser_block_means(K.cuda(), lengths=cuda(ints(lengths)), recent=recent, means=old.cuda()).cpu()
    want = ref.means(K, lengths, old, recent)
    untouched = want == old.double()
    # 64 additions in fp32 of values up to 5, and the rounding
    assert ((got.double() - want).abs() <= U[BF] * want.abs() + 64 * U[F32] * 5).all()
    assert torch.equal(got[untouched], old[untouched])


# ---------------------------------------------------------------- the choice of blocks
CASES = [
    # B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts
    (1, 1, 1, 1, 1, 1, 0, 1, True, None, None),
    (1, 2, 2, 200, 200, 2, 0, 1, True, None, None),
    (2, 6, 2, 130, 130, 3, 1, 1, False, None, None),
    (1, 8, 1, 3, 1000, 4, 1, 2, True, None, None),
    (3, 4, 2, 1, 777, 5, 0, 0, True, [1, 500, 777], None),
    (3, 4, 4, 150, 150, 2, 1, 1, True, [150, 0, 70], [0, 0, 0]),
    (2, 3, 1, 66, 500, 6, 2, 2, False, [500, 450], None),
    (2, 2, 1, 9, 2300, 33, 1, 1, True, [2300, 2111], None),
    (1, 10, 1, 40, 640, 8, 0, 1, True, None, None),
    (2, 2, 2, 5, 300, 64, 0, 1, True, [2, 300], None),       # fewer keys than queries; fewer blocks than places
    (2, 2, 2, 20, 400, 3, 0, 1, True, [400, 400], [-5, 390]),    # positions before the first key and behind the last
]


def inputs(case, seed=4):
    B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts = case
    gen = torch.Generator().manual_seed(seed)
    nb = -(-m // 64)
    lean = normal(gen, B, Hk, nb, 64, dtype=F32).repeat_interleave(64, 2)[:, :, :m]
    K = (normal(gen, B, Hk, m, 64, dtype=F32) + 0.4 * lean).to(BF)
    Q, V, D = normal(gen, B, Hq, n, 64), normal(gen, B, Hk, m, 64), normal(gen, B, Hq, n, 64)
    mean = ref.means(K, lengths, torch.full((B, Hk, nb, 64), math.nan), 0).to(BF)
    for b, x in enumerate(lengths or []):
        K[b, :, max(0, min(m, x)):] = math.nan               # behind a length nothing is read
        V[b, :, max(0, min(m, x)):] = math.inf
    return Q, K, V, D, mean


@pytest.mark.parametrize("case", CASES)
def test_select(dl, case):
    B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts = case
    Q, K, V, D, mean = inputs(case)
    got = dl.diffuser_select_blocks(Q.cuda(), mean.cuda(), top, keys=m, sink_blocks=sink, local_blocks=local,
                                    causal=causal, lengths=cuda(ints(lengths)), starts=cuda(ints(starts))).cpu()
    assert int((got != ref.select(Q, mean, top, m, sink, local, causal, lengths, starts)).sum()) == 0


@pytest.mark.parametrize("kind", ["zeros", "ties", "near", "nan", "inf", "huge", "tiny"])
@pytest.mark.parametrize("top", [1, 7, 40])
def test_select_hard_scores(dl, kind, top, n=20, nb=150):
    """Equal scores, scores that differ by less than fp32 sums resolve, and what is no number."""
    gen = torch.Generator().manual_seed(5)
    B, Hq, Hk = 1, 4, 2
    Q, mean = normal(gen, B, Hq, n, 64), normal(gen, B, Hk, nb, 64)
    if kind == "zeros":
        mean.zero_()
    if kind == "ties":
        mean[:, :, ::3] = mean[:, :, :1]
    if kind == "near":                                       # scores of +-2^20 that cancel but for one small product
        mean[..., 0], mean[..., 1] = 1024.0, -1024.0
        Q[..., 0] = Q[..., 1] = 1024.0
        mean[..., 2:] *= 2.0 ** -12
    if kind == "nan":
        mean[:, :, 5, 3] = math.nan
        Q[:, 0, 2] = math.nan
    if kind == "inf":
        mean[:, :, 5, 3], mean[:, :, 9, 4] = math.inf, -math.inf
    if kind == "huge":
        Q *= 1e20
        mean *= 1e18
    if kind == "tiny":
        Q *= 1e-25
        mean *= 1e-15
    got = dl.diffuser_select_blocks(Q.cuda(), mean.cuda(), top, keys=nb * 64 - 3, sink_blocks=1, local_blocks=0, causal=False).cpu()
    assert int((got != ref.select(Q, mean, top, nb * 64 - 3, 1, 0, False, None, None)).sum()) == 0


MANY = [   # enough queries for a thread each; the last tile short, more than a product's 128 blocks, many heads a group
    (1, 1, 1, 24650, 24650, 16, 1, 2, True, None, None),
    (2, 4, 2, 6200, 6200, 7, 0, 1, False, [6200, 1200], [0, 0]),
    (1, 12, 4, 6200, 20000, 20, 2, 1, True, None, None),
    (3, 30, 3, 2750, 3000, 4, 1, 1, True, [3000, 900, 0], None),
    (180, 2, 2, 70, 300, 3, 0, 0, False, None, None),
    (1, 1, 1, 24600, 40000, 1, 0, 0, False, None, None),
]


@pytest.mark.parametrize("case", MANY)
def test_select_many(dl, case):
    test_select(dl, case)


@pytest.mark.parametrize("kind", ["zeros", "ties", "near", "nan", "inf", "huge", "tiny"])
@pytest.mark.parametrize("top", [1, 7, 20, 32])
@pytest.mark.parametrize("nb", [150, 300])
def test_select_many_hard_scores(dl, kind, top, nb):
    test_select_hard_scores(dl, kind, top, n=12300, nb=nb)


@pytest.mark.parametrize("order", ["crowded", "rising", "falling"])
@pytest.mark.parametrize("top", [3, 12, 20])
@pytest.mark.parametrize("n,nb,G", [(9, 150, 2), (9, 900, 1), (25000, 300, 2), (25000, 600, 1)])
def test_select_uneven_scores(dl, order, top, n, nb, G):
    """The best blocks in four of 32 places, so that their maxima bound the choice badly, or in rising or falling order, so
    that the first to be looked at are the worst or the best of all."""
    gen = torch.Generator().manual_seed(7)
    Q, mean = normal(gen, 1, G, n, 64), normal(gen, 1, 1, nb, 64)
    Q[..., 0] = 4.0
    c = torch.arange(nb)
    mean[..., 0] = {"crowded": (c % 32 < 4) * 16.0, "rising": c * 1.0, "falling": (nb - c) * 1.0}[order]
    got = dl.diffuser_select_blocks(Q.cuda(), mean.cuda(), top, keys=nb * 64, sink_blocks=2, local_blocks=0, causal=False).cpu()
    assert torch.equal(got, ref.select(Q, mean, top, nb * 64, 2, 0, False, None, None))


# ---------------------------------------------------------------- attention
def attend(dl, case, Q, K, V, blocks, **kw):
    B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts = case
    return dl.diffuser_selected_attention(Q.cuda(), K.cuda(), V.cuda(), blocks.cuda(), causal=causal,
                                          lengths=cuda(ints(lengths)), starts=cuda(ints(starts)), **kw)


def check_attention(out, lse, Q, K, V, seen):
    want, sums, mass = ref.attend(Q, K, V, seen)
    # scores: 64 products in fp32, 2^-18 of sum |q k| / 8 at most, below 2^-12 here; the weights are rounded to bf16
    # for the product with V (2^-8 of each), and the result once
    assert ((out.double().cpu() - want).abs() <= U[BF] * want.abs() + (U[BF] + 2.0 ** -11) * mass).all()
    if lse is not None:
        empty = sums == -math.inf
        assert torch.equal(lse.cpu() == -math.inf, empty)
        assert ((lse.double().cpu() - sums).abs()[~empty] <= 2.0 ** -12 + 2.0 ** -22 * sums.abs()[~empty]).all()


@pytest.mark.parametrize("case", CASES)
def test_attention(dl, case):
    B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts = case
    Q, K, V, D, mean = inputs(case)
    blocks = ref.select(Q, mean, top, m, sink, local, causal, lengths, starts)
    seen = ref.mask(blocks, n, m, causal, lengths, starts)
    out, lse = attend(dl, case, Q, K, V, blocks, save_lse=True)
    check_attention(out, lse, Q, K, V, seen)
    assert torch.equal(attend(dl, case, Q, K, V, blocks), out)


def test_attention_lists(dl):
    """Lists of any values: repeated, falling, negative, too large, invisible, empty."""
    case = (1, 4, 2, 70, 330, 6, 0, 0, True, [329], None)
    Q, K, V, D, mean = inputs(case)
    gen = torch.Generator().manual_seed(6)
    blocks = torch.randint(-3, 9, (1, 2, 70, 6), generator=gen, dtype=torch.int32)
    blocks[:, :, 3] = -1
    blocks[:, :, 4] = 2 ** 31 - 1
    blocks[:, :, 5] = -2 ** 31
    blocks[:, :, 6] = torch.tensor([1, 1, 1, 1, 1, 1], dtype=torch.int32)
    blocks[:, :, 7] = torch.tensor([2 ** 31 - 1, 0, 1, 2, 3, 4], dtype=torch.int32)
    seen = ref.mask(blocks, 70, 330, True, [329], None)
    assert not seen[:, :, 7].any() and seen[:, :, 6].sum() == 128
    out, lse = attend(dl, case, Q, K, V, blocks, save_lse=True)
    check_attention(out, lse, Q, K, V, seen)


def check_gradients(got, Q, K, V, D, seen):
    want, mass, coarse, fine = ref.gradients(Q, K, V, D, seen)
    for y, w, a, c, f in zip(got, want, mass, coarse, fine):
        # the result's rounding; P's or dS's as an operand, and 2^-11 from the scores; delta's and dout.v's share
        bound = U[BF] * w.abs() + (U[BF] + 2.0 ** -11) * a + 1.1 * U[BF] * c + 2.0 ** -16 * f
        assert ((y.double().cpu() - w).abs() <= bound).all()


def backward(dl, case, Q, K, V, blocks, out, lse, D, **kw):
    B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts = case
    return dl.diffuser_selected_attention_backward(Q.cuda(), K.cuda(), V.cuda(), blocks.cuda(), out, lse, D.cuda(),
                                                   causal=causal, lengths=cuda(ints(lengths)), starts=cuda(ints(starts)), **kw)


# more rows than an item holds, lists of all lengths, heads that share a key block's items
LARGE = [
    (1, 2, 1, 1500, 1500, 4, 1, 1, True, None, None),
    (2, 2, 2, 1030, 1030, 5, 1, 2, False, [1030, 900], [0, 0]),
    (1, 16, 2, 300, 2000, 7, 2, 1, True, None, None),
    (1, 5, 1, 700, 700, 64, 0, 1, True, None, None),
]


@pytest.mark.parametrize("case", LARGE)
def test_attention_of_many_queries(dl, case):
    B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts = case
    Q, K, V, D, mean = inputs(case)
    blocks = dl.diffuser_select_blocks(Q.cuda(), mean.cuda(), top, keys=m, sink_blocks=sink, local_blocks=local,
                                       causal=causal, lengths=cuda(ints(lengths)), starts=cuda(ints(starts))).cpu()
    assert torch.equal(blocks, ref.select(Q, mean, top, m, sink, local, causal, lengths, starts))
    seen = ref.mask(blocks, n, m, causal, lengths, starts)
    out, lse = attend(dl, case, Q, K, V, blocks, save_lse=True)
    check_attention(out, lse, Q, K, V, seen)
    assert torch.equal(attend(dl, case, Q, K, V, blocks), out)
    got = backward(dl, case, Q, K, V, blocks, out, lse, D)
    check_gradients(got, Q, K, V, D, seen)
    for x, y in zip(got, backward(dl, case, Q, K, V, blocks, out, lse, D)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("case", [(1, 1, 1, 3900, 17000, 6, 1, 1, True, [16900], None), (1, 1, 1, 4100, 16450, 3, 0, 1, False, None, None)])
def test_attention_of_many_queries_and_blocks(dl, case):
    """More key blocks than one block of threads sums up at a time, and as many chunks of queries."""
    test_attention_of_many_queries(dl, case)


@pytest.mark.parametrize("case", CASES)
def test_backward(dl, case):
    B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts = case
    Q, K, V, D, mean = inputs(case)
    blocks = ref.select(Q, mean, top, m, sink, local, causal, lengths, starts)
    out, lse = attend(dl, case, Q, K, V, blocks, save_lse=True)
    check_gradients(backward(dl, case, Q, K, V, blocks, out, lse, D), Q, K, V, D, ref.mask(blocks, n, m, causal, lengths, starts))
