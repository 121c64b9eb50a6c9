"""The rotation alone and the attention over chosen key blocks at the limits of what they promise,
against their definitions in 64 bits."""
import math

import pytest
import torch

from tests import selected_reference as ref
from tests.test_gpu_selected import attend, backward, check_attention, check_gradients, inputs
from tests import test_gpu_selected as plain

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8                                                # half a bf16 step


@pytest.fixture(scope="module")
def dl():
    from sparse_long_sequence_gb300 import binding
    return binding


# ---------------------------------------------------------------- the weights of the attention
@pytest.mark.parametrize("B,Hq,Hk,n,m,top,causal,few", [
    (2, 8, 2, 3, 600, 5, True, True), (1, 16, 1, 1, 900, 9, False, True), (3, 2, 2, 40, 40, 3, True, True),
    (1, 4, 2, 1500, 1500, 6, True, False), (2, 3, 1, 1100, 1200, 7, False, False)])
def test_weights_keep_more_than_an_operands_bits(dl, B, Hq, Hk, n, m, top, causal, few):
    """Scores that fp32 sums hold exactly, so that the weights' own error shows."""
    gen = torch.Generator().manual_seed(1)
    Q = torch.randint(-2, 3, (B, Hq, n, 64), generator=gen).to(BF)
    K = (torch.randint(-2, 3, (B, Hk, m, 64), generator=gen) * 0.25).to(BF)
    V = torch.randn((B, Hk, m, 64), generator=gen).to(BF)
    mean = ref.means(K, None, torch.zeros((B, Hk, -(-m // 64), 64)), 0).to(BF)
    blocks = ref.select(Q, mean, top, m, 0, 1, causal, None, None)
    assert (dl.diffuser_selected_attention_workspace_size(B, Hq, Hk, n, m, top) == 0) == few
    out = dl.diffuser_selected_attention(Q.cuda(), K.cuda(), V.cuda(), blocks.cuda(), causal=causal)
    want, _, mass = ref.attend(Q, K, V, ref.mask(blocks, n, m, causal, None, None))
    # of a weight: its low part, below 2^-7 of it, is rounded by 2^-8 of itself, 2^-15; 2^-22 on top of it; the
    # exponential and its argument below 2^-18.  Of the sums: eight products of 16 terms with 17 2^-23 each, and the
    # joining below 2^-20.  Together 5.2e-5, below 2^-14; and the result's rounding
    assert ((out.double().cpu() - want).abs() <= U * want.abs() + 2.0 ** -14 * mass).all()


def test_an_infinite_value_stays_one(dl):
    """Rows that see one infinite value have it in their results, with its sign."""
    gen = torch.Generator().manual_seed(2)
    for n in (4, 800):
        Q, K, V = (torch.randn((1, 2, x, 64), generator=gen).to(BF) for x in (n, 640, 640))
        blocks = torch.arange(10, dtype=torch.int32).expand(1, 2, n, 10).contiguous()
        V[0, 0, 5, 7], V[0, 1, 600, 63] = math.inf, -math.inf
        few = dl.diffuser_selected_attention_workspace_size(1, 2, 2, n, 640, 10) == 0
        assert few == (n == 4)
        out = dl.diffuser_selected_attention(Q.cuda(), K.cuda(), V.cuda(), blocks.cuda(), causal=False).cpu()
        want = torch.zeros_like(out)
        some = slice(max(0, n - 640), n)                     # (more queries than keys: the first ones see none)
        want[0, 0, some, 7], want[0, 1, some, 63] = math.inf, -math.inf
        assert torch.equal(torch.where(out.isinf(), out, 0.0), want) and not out.isnan().any()


# ---------------------------------------------------------------- the rotation
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rot", [16, 32, 48])
@pytest.mark.parametrize("inter", [False, True])
def test_features_that_are_not_turned_are_copied(dl, dtype, rot, inter):
    """Bit by bit, whatever they are, and nothing of them reaches the others."""
    gen = torch.Generator().manual_seed(3)
    word = torch.int16 if dtype == BF else torch.int32
    q, k = (torch.randn((2, h, 37, 64), generator=gen).to(dtype) for h in (3, 1))
    freq, mag = dl.diffuser_rope_frequencies(rot, 10000.0, dl.DIFFUSER_ROPE_YARN, 4.0, 4096)
    top = 0x7f80 << (0 if dtype == BF else 16)               # infinity's bits; above them NaN
    sign = -(1 << (15 if dtype == BF else 31))
    odd = torch.tensor([top, top + sign, top + 1, top + 3, 1, sign, -1])     # infinities, NaN, the least value, -0, NaN
    for call, names in ((dl.diffuser_rope, ("Qo", "Ko")), (dl.diffuser_rope_backward, ("dQ", "dK"))):
        plain = call(q.cuda(), k.cuda(), freq, magnitude=mag, interleaved=inter)
        marked = []
        for x in (q, k):
            y = x.clone()
            bits = odd[torch.randint(0, 7, y[..., rot:].shape, generator=gen)].to(word)
            y[..., rot:] = torch.where(torch.rand(bits.shape, generator=gen) < 0.5, bits.view(dtype), y[..., rot:])
            marked.append(y.cuda())
        got = call(*marked, freq, magnitude=mag, interleaved=inter)
        for x, y, z in zip(marked, got, plain):
            assert torch.equal(x[..., rot:].contiguous().view(word), y[..., rot:].contiguous().view(word))
            assert torch.equal(y[..., :rot].contiguous().view(word), z[..., :rot].contiguous().view(word))
        same = call(*marked, freq, magnitude=mag, interleaved=inter, **dict(zip(names, marked)))
        for x, y in zip(same, got):
            assert torch.equal(x.view(word), y.view(word))


# ---------------------------------------------------------------- the choice of blocks
LEAST = 2.0 ** -133                                          # bf16's least value


@pytest.mark.parametrize("kind", ["least queries", "least means beside a large one", "both"])
@pytest.mark.parametrize("top", [1, 7, 20, 40])
@pytest.mark.parametrize("n,nb", [(300, 150), (12300, 150), (12300, 300)])
def test_choice_by_products_below_fp32s_range(dl, kind, top, n, nb):
    """Products of 2^-143 and less, which fp32 has to round; in 64 bits scores are exact."""
    gen = torch.Generator().manual_seed(4)
    Hq, Hk = 4, 2
    whole = lambda *s: torch.randint(-7, 8, s, generator=gen, dtype=torch.float64) * LEAST
    Q, mean = torch.randn((1, Hq, n, 64), generator=gen) * 1e-3, torch.randn((1, Hk, nb, 64), generator=gen) * 1e-3
    if kind != "least means beside a large one":
        Q = whole(1, Hq, n, 64)
    if kind != "least queries":
        mean = whole(1, Hk, nb, 64)
        mean[:, :, 0] = 1.0
    Q, mean = Q.to(BF), mean.to(BF)
    got = dl.diffuser_select_blocks(Q.cuda(), mean.cuda(), top, keys=nb * 64, sink_blocks=1, local_blocks=0, causal=False).cpu()
    assert torch.equal(got, ref.select(Q, mean, top, nb * 64, 1, 0, False, None, None))


# ---------------------------------------------------------------- the attention of many sequences' tokens
@pytest.mark.parametrize("n", [1, 3])
def test_tokens_of_a_large_batch(dl, n):
    """160 sequences of 8 key heads: no workspace, and each as it is by itself."""
    B, Hq, Hk, m, top = 160, 32, 8, 700, 9
    rand = lambda seed, *s: torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)
    q, k, v = rand(1, B, Hq, n, 64), rand(2, B, Hk, m, 64), rand(3, B, Hk, m, 64)
    lengths = (torch.arange(B, device="cuda") * 37 % (m + 1)).to(torch.int32)
    blocks = dl.diffuser_select_blocks(q, dl.diffuser_block_means(k, lengths=lengths), top, keys=m, lengths=lengths)
    assert dl.diffuser_selected_attention_workspace_size(B, Hq, Hk, n, m, top) == 0
    out, lse = dl.diffuser_selected_attention(q, k, v, blocks, lengths=lengths, save_lse=True)
    for b in (0, 1, 77, 159):
        one = [x[b:b + 1].contiguous() for x in (q, k, v, blocks)]
        o, l = dl.diffuser_selected_attention(*one, lengths=lengths[b:b + 1].clone(), save_lse=True)
        assert torch.equal(o[0], out[b]) and torch.equal(l[0], lse[b])
        seen = ref.mask(one[3].cpu(), n, m, True, [int(lengths[b])], None)
        want, sums, mass = ref.attend(*(x.cpu() for x in one[:3]), seen)
        # 2^-11 of a weight from its score's fp32 sum, 2^-14 from its parts and the sums (above)
        assert ((o.double().cpu() - want).abs() <= U * want.abs() + 2.0 ** -10 * mass).all()


def test_many_queries_that_list_nothing(dl):
    """By block: no tiles at all, or none but one head's."""
    n, top = 800, 12
    rand = lambda seed, *s: torch.randn(s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)
    q, k, v, d = rand(1, 1, 4, n, 64), rand(2, 1, 2, n, 64), rand(3, 1, 2, n, 64), rand(4, 1, 4, n, 64)
    assert dl.diffuser_selected_attention_workspace_size(1, 4, 2, n, n, top) > 0
    none = torch.full((1, 2, n, top), -1, dtype=torch.int32, device="cuda")
    some = none.clone()
    some[0, 1, :, 0] = 0
    for blocks in (none, some):
        out, lse = dl.diffuser_selected_attention(q, k, v, blocks, causal=False, save_lse=True)
        dq, dk, dv = dl.diffuser_selected_attention_backward(q, k, v, blocks, out, lse, d, causal=False)
        seen = ref.mask(blocks.cpu(), n, n, False, None, None)
        want, sums, mass = ref.attend(q.cpu(), k.cpu(), v.cpu(), seen)
        assert ((out.double().cpu() - want).abs() <= U * want.abs() + 2.0 ** -10 * mass).all()
        assert torch.equal(lse.cpu() == -math.inf, sums == -math.inf)
        assert not dq[0, :2].any() and not dk[0, 0].any() and not dv[0, 0].any() and not dk[0, 1, 64:].any()
        assert bool(dv[0, 1, :64].any()) == (blocks is some)


@pytest.mark.parametrize("B,Hq,Hk,n,m,top,sink,local,causal,lengths,starts", [
    (1, 40, 1, 24700, 6400, 9, 1, 1, False, None, None),     # many heads a group, few and many key blocks
    (2, 32, 1, 12500, 33000, 5, 0, 1, True, [33000, 20000], None),
    (1, 24, 1, 74000, 1500, 3, 0, 1, True, None, None),
    (1, 8, 2, 12400, 9600, 21, 1, 2, True, None, None),      # more blocks than a thread's list serves
    (3, 12, 3, 2800, 4000, 32, 2, 1, True, [4000, 900, 3333], None),
    (1, 4, 1, 24700, 9600, 33, 0, 1, False, [9555], None)])
def test_choice_for_many_queries_of_grouped_heads(dl, B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts):
    gen = torch.Generator().manual_seed(5)
    Q, mean = torch.randn((B, Hq, n, 64), generator=gen).to(BF), torch.randn((B, Hk, -(-m // 64), 64), generator=gen).to(BF)
    given = [None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lengths, starts)]
    got = dl.diffuser_select_blocks(Q.cuda(), mean.cuda(), top, keys=m, sink_blocks=sink, local_blocks=local, causal=causal,
                                    lengths=given[0], starts=given[1]).cpu()
    assert torch.equal(got, ref.select(Q, mean, top, m, sink, local, causal, lengths, starts))


# ---------------------------------------------------------------- lists of any values
def any_lists(gen, B, Hk, n, top, nb):
    """Falling, repeated, negative, too large, empty; and some as a choice would give them."""
    blocks = torch.randint(-3, nb + 3, (B, Hk, n, top), generator=gen, dtype=torch.int32)
    kind = torch.randint(0, 8, (B, Hk, n, 1), generator=gen)
    blocks = torch.where(kind < 3, blocks.sort(-1).values, blocks)
    blocks = torch.where(kind == 3, blocks.sort(-1, descending=True).values, blocks)
    blocks = torch.where(kind == 4, blocks[..., :1], blocks)
    blocks[:, :, 3::50] = -1
    blocks[:, :, 4::50] = 2 ** 31 - 1
    blocks[:, :, 5::50] = -2 ** 31
    blocks[:, :, 6::50, 1:] = torch.arange(top - 1, dtype=torch.int32)
    blocks[:, :, 6::50, 0] = 2 ** 31 - 1                     # nothing is above the first entry
    blocks[:, :, 7::50] = torch.arange(top, dtype=torch.int32)
    blocks[:, :, 7::50, top // 2] = -2 ** 31                 # one that does not count between those that do
    return blocks


@pytest.mark.parametrize("B,Hq,Hk,n,m,top,causal,lengths,starts", [
    (2, 2, 2, 1200, 1100, 3, True, [1100, 700], [-20, 0]), (1, 4, 4, 1200, 1100, 4, False, None, None),
    (2, 6, 2, 1200, 1100, 7, True, [1099, 1], [0, 0]), (1, 3, 1, 1200, 1100, 16, True, None, [0]),
    (1, 16, 2, 1200, 1100, 12, True, [1000], [0]), (1, 4, 2, 1200, 1100, 33, False, [1090], [0]),
    (1, 2, 2, 1200, 1100, 64, True, None, [0]), (1, 4, 2, 70, 330, 6, True, [329], None), (2, 9, 1, 5, 1000, 61, False, None, None)])
def test_any_lists(dl, B, Hq, Hk, n, m, top, causal, lengths, starts):
    case = (B, Hq, Hk, n, m, top, 0, 0, causal, lengths, starts)
    Q, K, V, D, _ = inputs(case)
    blocks = any_lists(torch.Generator().manual_seed(6), B, Hk, n, top, -(-m // 64))
    assert (dl.diffuser_selected_attention_workspace_size(B, Hq, Hk, n, m, top) > 0) == (n == 1200)
    seen = ref.mask(blocks, n, m, causal, lengths, starts)
    out, lse = attend(dl, case, Q, K, V, blocks, save_lse=True)
    check_attention(out, lse, Q, K, V, seen)
    grads = backward(dl, case, Q, K, V, blocks, out, lse, D)
    check_gradients(grads, Q, K, V, D, seen)
    assert torch.equal(attend(dl, case, Q, K, V, blocks), out)
    assert all(torch.equal(x, y) for x, y in zip(grads, backward(dl, case, Q, K, V, blocks, out, lse, D)))


@pytest.mark.parametrize("B,Hq,Hk,n,m,top,sink,local,causal,lengths,starts", [
    (1, 16, 2, 900, 2000, 7, 2, 1, True, None, None), (1, 2, 1, 3000, 3000, 5, 1, 1, True, None, None)])
def test_tiles_of_grouped_heads(dl, B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts):
    assert dl.diffuser_selected_attention_workspace_size(B, Hq, Hk, n, m, top) > 0
    plain.test_attention_of_many_queries(dl, (B, Hq, Hk, n, m, top, sink, local, causal, lengths, starts))


# ---------------------------------------------------------------- positions of the rotation
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("offset", [0, 1, 777, -5, 3 * 2 ** 20, 2 ** 45 + 12345, -2 ** 33])
def test_offsets_and_positions_add_up(dl, offset, inter):
    """An offset alone, and one with positions, against the definition at their sums."""
    gen = torch.Generator().manual_seed(7)
    B, n = 2, 21
    q, k = torch.randn((B, 3, n, 64), generator=gen), torch.randn((B, 2, n, 64), generator=gen)
    freq, mag = dl.diffuser_rope_frequencies(48, 10000.0, dl.DIFFUSER_ROPE_YARN, 4.0, 4096)
    own = torch.arange(n).expand(B, n)
    given = torch.randint(-1000, 1 << 20, (B, n), generator=gen)
    for call, sign in ((dl.diffuser_rope, 1), (dl.diffuser_rope_backward, -1)):
        for pos, at in ((None, own), (given, given)):
            how = dict(magnitude=mag, interleaved=inter)
            got = call(q.cuda(), k.cuda(), freq, positions=None if pos is None else pos.cuda(), position_offset=offset, **how)
            same = call(q.cuda(), k.cuda(), freq, positions=(at + offset).cuda(), **how)
            assert all(torch.equal(x, y) for x, y in zip(got, same))
            if abs(offset) > 1 << 32:
                continue                                     # (the reference's angles lose their fractions there)
            for x, y in zip((q, k), got):
                want = ref.rope(x, freq, mag, inter, sign * (at + offset))
                # a cosine's argument is off by 2^-31 turns and its value by 2^-23, the reference's by 2^-53 of 2^22 radians;
                # three fp32 operations
                pair = 2.0 ** -20 * mag * x.double().abs().amax(-1, keepdim=True)
                assert ((y.double().cpu() - want).abs() <= 2.0 ** -24 * want.abs() + pair).all()
