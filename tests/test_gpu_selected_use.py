"""The operators of the attention over chosen key blocks as they are used: together, captured into
graphs, on streams, with outputs in the middle of other data, on caches past 2^31 elements, on more
queries than the workspace holds partial sums of at once; and their refusals."""
import math
import os
import subprocess
import sys

import pytest
import torch

from tests import selected_reference as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -8                                                # half a bf16 step


@pytest.fixture(scope="module")
def dl():
    from sparse_long_sequence_gb300 import binding
    return binding


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF)


def step(dl, q, k, v, freq, mag, top, dout=None, **how):
    """Rotation, means, choice, attention and (dout) the gradients of what went in."""
    qr, kr = dl.diffuser_rope(q, k, freq, magnitude=mag)
    mean = dl.diffuser_block_means(kr, lengths=how.get("lengths"))
    blocks = dl.diffuser_select_blocks(qr, mean, top, keys=k.shape[2], sink_blocks=1, **how)
    out, lse = dl.diffuser_selected_attention(qr, kr, v, blocks, save_lse=True, **how)
    if dout is None:
        return [qr, kr, mean, blocks, out, lse]
    dqr, dkr, dv = dl.diffuser_selected_attention_backward(qr, kr, v, blocks, out, lse, dout, **how)
    dq, dk = dl.diffuser_rope_backward(dqr, dkr, freq, magnitude=mag)
    return [qr, kr, mean, blocks, out, lse, dq, dk, dv]


def test_together(dl):
    """A training step of the whole chain against automatic differentiation in 64 bits."""
    B, Hq, Hk, n, top = 2, 4, 2, 700, 4
    q, k, v, dout = rand(1, B, Hq, n, 64), rand(2, B, Hk, n, 64), rand(3, B, Hk, n, 64), rand(4, B, Hq, n, 64)
    freq, mag = dl.diffuser_rope_frequencies(64, 10000.0, dl.DIFFUSER_ROPE_YARN, 4.0, 4096)
    qr, kr, mean, blocks, out, lse, dq, dk, dv = (x.cpu() for x in step(dl, q, k, v, freq, mag, top, dout))
    # each stage from what the one before gave: the choice is exact, so no gap opens
    pos = torch.arange(n).expand(B, n)
    assert ((qr.double() - ref.rope(q.cpu(), freq, mag, False, pos)).abs() <= U * qr.double().abs() + 2.0 ** -16).all()
    assert torch.equal(blocks, ref.select(qr, mean, top, n, 1, 1, True, None, None))
    seen = ref.mask(blocks, n, n, True, None, None)
    want, sums, mass = ref.attend(qr, kr, v.cpu(), seen)
    assert ((out.double() - want).abs() <= U * want.abs() + (U + 2.0 ** -11) * mass).all()
    assert ((lse.double() - sums).abs() <= 2.0 ** -12 + 2.0 ** -22 * sums.abs()).all()
    a, b, c = (x.cpu().double().requires_grad_(True) for x in (q, k, v))
    ar, br = ref.rope(a, freq, mag, False, pos), ref.rope(b, freq, mag, False, pos)
    x = (ar @ br.repeat_interleave(2, 1).mT / 8).masked_fill(~seen.repeat_interleave(2, 1), -math.inf)
    y = torch.softmax(x, -1) @ c.repeat_interleave(2, 1)
    grads = torch.autograd.grad(y, (a, b, c), dout.cpu().double())
    for got, g in zip((dq, dk, dv), grads):
        # the roundings of q, k and out to bf16 between the stages, of P and dS as operands, of each result: seven
        # half steps, random and independent, of terms whose sum is up to four times the result in the 2-norm
        assert float((got.double() - g).norm()) <= 4 * math.sqrt(7) * U * float(g.norm())


def test_gradients_against_differences(dl):
    """The change of <dout, out> along a direction, by central differences in 64 bits on the chosen blocks."""
    B, Hq, Hk, n, top = 1, 2, 1, 300, 3
    q, k, v, dout = (rand(s, B, h, n, 64) for s, h in ((5, Hq), (6, Hk), (7, Hk), (8, Hq)))
    mean = dl.diffuser_block_means(k)
    blocks = dl.diffuser_select_blocks(q, mean, top, keys=n)
    out, lse = dl.diffuser_selected_attention(q, k, v, blocks, save_lse=True)
    grads = dl.diffuser_selected_attention_backward(q, k, v, blocks, out, lse, dout)
    seen = ref.mask(blocks.cpu(), n, n, True, None, None).repeat_interleave(2, 1).cuda()

    def value(x):
        a, b, c = x
        s = (a @ b.repeat_interleave(2, 1).mT / 8).masked_fill(~seen, -math.inf)
        return float((torch.softmax(s, -1) @ c.repeat_interleave(2, 1) * dout.double()).sum())
    at = [x.double() for x in (q, k, v)]
    for which, grad in enumerate(grads):
        g = torch.Generator(device="cuda").manual_seed(9 + which)
        d = torch.randn(at[which].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        ends = []
        for sign in (1, -1):
            x = list(at)
            x[which] = x[which] + sign * h * d
            ends.append(value(x))
        slope = (ends[0] - ends[1]) / (2 * h)
        terms = grad.double() * d
        # each gradient is off by a few half steps of its own size, at random: 6 U of the terms' 2-norm
        assert abs(float(terms.sum()) - slope) <= 6 * U * float(terms.norm()) + 1e-6 * abs(slope)


def serve(dl, cache_k, cache_v, mean, q, lengths, top):
    dl.diffuser_block_means(cache_k, lengths=lengths, recent=1, means=mean)
    blocks = dl.diffuser_select_blocks(q, mean, top, keys=cache_k.shape[2], sink_blocks=1, local_blocks=2, lengths=lengths)
    return dl.diffuser_selected_attention(q, cache_k, cache_v, blocks, lengths=lengths)


def test_serving_steps_give_what_the_prompt_gives(dl):
    """Tokens appended one at a time to caches of different lengths, captured and replayed, against the whole
    sequences at once: the same choices, and results within their roundings."""
    B, Hq, Hk, cap, top, steps = 3, 4, 2, 512, 3, 70
    first = torch.tensor([1, 60, 300], dtype=torch.int32, device="cuda")
    K, V, Q = rand(10, B, Hk, cap, 64), rand(11, B, Hk, cap, 64), rand(12, B, Hq, cap, 64)
    length = first.clone()
    mean = dl.diffuser_block_means(K, lengths=length)
    q = torch.empty((B, Hq, 1, 64), dtype=BF, device="cuda")
    rows = torch.arange(B, device="cuda")

    def next_token():
        length.add_(1)
        q.copy_(Q[rows, :, length.long() - 1].unsqueeze(2))
        return serve(dl, K, V, mean, q, length, top)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = next_token()
    got = []
    for _ in range(steps):
        graph.replay()
        got.append(out.clone())
    torch.cuda.synchronize()
    assert torch.equal(length, first + steps)
    for b in range(B):
        m = int(length[b])
        k, v, qs = K[b:b + 1, :, :m].contiguous(), V[b:b + 1, :, :m].contiguous(), Q[b:b + 1, :, :m].contiguous()
        # a block's mean changes while it fills, so each step is chosen on the keys up to its own
        for t in (0, 3, 40, steps - 1):
            at = int(first[b]) + t
            kt, vt, qt = k[:, :, :at + 1].contiguous(), v[:, :, :at + 1].contiguous(), qs[:, :, at:at + 1].contiguous()
            blocks = ref.select(qt.cpu(), dl.diffuser_block_means(kt).cpu(), top, at + 1, 1, 2, True, None, None)
            want, _, mass = ref.attend(qt.cpu(), kt.cpu(), vt.cpu(), ref.mask(blocks, 1, at + 1, True, None, None))
            y = got[t][b:b + 1].double().cpu()
            assert ((y - want).abs() <= U * want.abs() + (U + 2.0 ** -11) * mass).all()


SIZES = [(2, 4, 2, 40, 4), (1, 6, 2, 1500, 6)]               # by query, and by block


@pytest.mark.parametrize("B,Hq,Hk,n,top", SIZES)
def test_captured_graphs_and_streams(dl, B, Hq, Hk, n, top):
    freq, mag = dl.diffuser_rope_frequencies(64, 10000.0, dl.DIFFUSER_ROPE_NTK, 4.0)
    sets = [[rand(s + 20 * k, B, h, n, 64) for s, h in ((1, Hq), (2, Hk), (3, Hk), (4, Hq))] for k in range(2)]
    want = [step(dl, q, k, v, freq, mag, top, d) for q, k, v, d in sets]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for (q, k, v, d), s in zip(sets, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(step(dl, q, k, v, freq, mag, top, d))
        graphs.append(g)
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    # eager calls at once on two streams, and one given its stream
    got = [[], []]
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(step(dl, *sets[k][:3], freq, mag, top, sets[k][3]))
    torch.cuda.synchronize()
    for runs, w in zip(got, want):
        assert all(torch.equal(a, b) for r in runs for a, b in zip(r, w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q, k, v, d = sets[0]
    y = dl.diffuser_selected_attention(want[0][0], want[0][1], v, want[0][3], stream=s)
    s.synchronize()
    assert torch.equal(y, want[0][4])


@pytest.mark.parametrize("n", [3, 900, 24700])
def test_first_call_inside_a_capture(dl, n):
    code = f"""
import torch
from sparse_long_sequence_gb300 import binding as dl
r = lambda h: torch.randn(1, h, {n}, 64, device='cuda').bfloat16()
q, k, v, d = r(2), r(1), r(1), r(2)
torch.cuda.synchronize()
def run():
    f, m = dl.diffuser_rope_frequencies()
    a, b = dl.diffuser_rope(q, k, f)
    mean = dl.diffuser_block_means(b)
    blocks = dl.diffuser_select_blocks(a, mean, 5, keys={n})
    o, l = dl.diffuser_selected_attention(a, b, v, blocks, save_lse=True)
    return [a, b, mean, blocks, o, l, *dl.diffuser_selected_attention_backward(a, b, v, blocks, o, l, d)]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, run()))
print('fine')
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("n,m", [(3, 500), (1300, 1300)])
def test_nothing_is_written_outside(dl, n, m):
    """Outputs and the workspace between guards; a workspace that holds other bits gives the same."""
    B, Hq, Hk, top = 2, 6, 3, 5
    q, k, v, d = rand(30, B, Hq, n, 64), rand(31, B, Hk, m, 64), rand(32, B, Hk, m, 64), rand(33, B, Hq, n, 64)
    guarded = []

    def guard(shape, dtype, fill):
        size = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        room = torch.full((size + 2048,), fill, dtype=torch.uint8, device="cuda")
        start = 1024 - room.data_ptr() % 256
        guarded.append((room, start, size, fill))
        return room[start:start + size].view(dtype).view(shape)
    seen = []
    for fill in (0x5a, 0xff):
        mean = guard((B, Hk, -(-m // 64), 64), BF, fill)
        dl.diffuser_block_means(k, means=mean)
        blocks = guard((B, Hk, n, top), torch.int32, fill)
        dl.diffuser_select_blocks(q, mean, top, keys=m, blocks=blocks)
        out, lse = guard(q.shape, BF, fill), guard((B, Hq, n), torch.float32, fill)
        size = dl.diffuser_selected_attention_workspace_size(B, Hq, Hk, n, m, top)
        ws = guard((max(size, 1),), torch.uint8, fill)
        dl.diffuser_selected_attention(q, k, v, blocks, out=out, lse=lse, workspace=ws)
        grads = [guard(x.shape, BF, fill) for x in (q, k, v)]
        ws2 = guard((dl.diffuser_selected_attention_backward_workspace_size(B, Hq, Hk, n, m, top),), torch.uint8, fill)
        dl.diffuser_selected_attention_backward(q, k, v, blocks, out, lse, d, dQ=grads[0], dK=grads[1], dV=grads[2], workspace=ws2)
        seen.append([x.clone() for x in (mean, blocks, out, lse, *grads)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*seen))
    for room, start, size, fill in guarded:
        assert (room[:start] == fill).all() and (room[start + size:] == fill).all()


def test_caches_past_32_bits(dl):
    """2.2e9 elements of keys and of values: the last sequence's step."""
    B, Hk, m, top = 34, 1, 1 << 20, 6
    K = torch.zeros((B, Hk, m, 64), dtype=BF, device="cuda")
    V = torch.zeros_like(K)
    K[-1], V[-1] = rand(40, Hk, m, 64), rand(41, Hk, m, 64)
    q = rand(42, B, 2, 1, 64)
    mean = dl.diffuser_block_means(K)
    blocks = dl.diffuser_select_blocks(q, mean, top, keys=m, sink_blocks=1, local_blocks=1)
    out = dl.diffuser_selected_attention(q, K, V, blocks)
    last = [x[-1:].contiguous() for x in (q, K, V)]
    m1 = dl.diffuser_block_means(last[1])
    b1 = dl.diffuser_select_blocks(last[0], m1, top, keys=m, sink_blocks=1, local_blocks=1)
    assert torch.equal(mean[-1:], m1) and torch.equal(blocks[-1:], b1)
    assert torch.equal(out[-1:], dl.diffuser_selected_attention(*last, b1))
    assert not out[:-1].any()
    want = torch.einsum("hnd,cd->nc", last[0][0].double(), m1[0, 0].double())[0]
    want[0] = want[-1] = math.inf
    assert torch.equal(b1[0, 0, 0].long(), want.topk(top).indices.sort().values)


def test_many_units_in_groups(dl):
    """More partial sums than the workspace holds at once: the same as the sequences one by one."""
    B, H, n, top = 5, 4, 16384, 16
    q, k, v, d = (rand(50 + s, B, H, n, 64) for s in range(4))
    size = dl.diffuser_selected_attention_workspace_size(B, H, H, n, n, top)
    assert size < 2 * dl.diffuser_selected_attention_workspace_size(B - 1, H, H, n, n, top)
    mean = dl.diffuser_block_means(k)
    blocks = dl.diffuser_select_blocks(q, mean, top, keys=n, sink_blocks=1, local_blocks=2)
    out, lse = dl.diffuser_selected_attention(q, k, v, blocks, save_lse=True)
    grads = dl.diffuser_selected_attention_backward(q, k, v, blocks, out, lse, d)
    again = dl.diffuser_selected_attention_backward(q, k, v, blocks, out, lse, d)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    for b in (0, B - 1):
        one = [x[b:b + 1].contiguous() for x in (q, k, v, blocks, d)]
        o, l = dl.diffuser_selected_attention(*one[:4], save_lse=True)
        assert torch.equal(o[0], out[b]) and torch.equal(l[0], lse[b])
        g = dl.diffuser_selected_attention_backward(*one[:4], o, l, one[4])
        assert torch.equal(g[0][0], grads[0][b])             # (dk and dv are added up in other runs of tiles)
        for x, y in zip(g[1:], grads[1:]):
            # two fp32 sums in another order, each rounded once: a step of bf16 apart, and 2^-20 of the largest
            x, y = x[0].double(), y[b].double()
            assert ((x - y).abs() <= 2 * U * x.abs() + 2.0 ** -20 * x.abs().max()).all()
    # a few rows against the definition
    h, rows = 2, [0, 63, 64, 5000, 16383]
    for i in rows:
        keys = torch.cat([torch.arange(c * 64, min(c * 64 + 64, i + 1)) for c in blocks[4, h, i].tolist() if c >= 0]).cuda()
        p = torch.softmax(q[4, h, i].double() @ k[4, h, keys].double().T / 8, 0)
        want = p @ v[4, h, keys].double()
        mass = p @ v[4, h, keys].double().abs()
        assert ((out[4, h, i].double() - want).abs() <= U * want.abs() + (U + 2.0 ** -11) * mass).all()


def test_refusals_of_the_binding(dl):
    q, k = rand(60, 1, 4, 20, 64), rand(61, 1, 2, 100, 64)
    mean = dl.diffuser_block_means(k)
    blocks = dl.diffuser_select_blocks(q, mean, 2, keys=100)
    out, lse = dl.diffuser_selected_attention(q, k, k, blocks, save_lse=True)
    freq, _ = dl.diffuser_rope_frequencies()
    i32 = torch.tensor([50], dtype=torch.int32, device="cuda")
    before = dl.diffuser_launch_count()[0]
    bad = [lambda: dl.diffuser_rope(q, q.float(), freq), lambda: dl.diffuser_rope(q, k, freq),
           lambda: dl.diffuser_rope(q, q.clone(), list(freq)[:5]), lambda: dl.diffuser_rope(q, q.clone(), []),
           lambda: dl.diffuser_rope(q, q.clone(), freq, magnitude=0.0), lambda: dl.diffuser_rope(q, q.clone(), freq, Qo=q, Ko=q),
           lambda: dl.diffuser_rope(q, q.clone(), freq, positions=i32), lambda: dl.diffuser_rope(q.cpu(), q, freq),
           lambda: dl.diffuser_rope_frequencies(100), lambda: dl.diffuser_rope_frequencies(24),
           lambda: dl.diffuser_rope_frequencies(64, 0.5), lambda: dl.diffuser_rope_frequencies(64, 1e4, 7),
           lambda: dl.diffuser_block_means(k.float()), lambda: dl.diffuser_block_means(k[0]),
           lambda: dl.diffuser_block_means(k.transpose(1, 2)), lambda: dl.diffuser_block_means(k, recent=-1),
           lambda: dl.diffuser_block_means(k, lengths=i32.long()), lambda: dl.diffuser_block_means(k, lengths=i32.repeat(2)),
           lambda: dl.diffuser_block_means(k, means=mean[:, :, :1]), lambda: dl.diffuser_block_means(k[..., :32].contiguous()),
           lambda: dl.diffuser_select_blocks(q, mean, 0, keys=100), lambda: dl.diffuser_select_blocks(q, mean, 65, keys=100),
           lambda: dl.diffuser_select_blocks(q, mean, 2, keys=300), lambda: dl.diffuser_select_blocks(q, mean, 2, keys=100, sink_blocks=2),
           lambda: dl.diffuser_select_blocks(q[:, :3].contiguous(), mean, 2, keys=100),
           lambda: dl.diffuser_select_blocks(q.float(), mean, 2, keys=100), lambda: dl.diffuser_select_blocks(q, mean.cpu(), 2, keys=100),
           lambda: dl.diffuser_select_blocks(q, mean, 2, keys=100, starts=i32.cpu()),
           lambda: dl.diffuser_select_blocks(q, mean, 2, keys=100, blocks=blocks.long()),
           lambda: dl.diffuser_selected_attention(q, k, k[:, :, :50], blocks), lambda: dl.diffuser_selected_attention(q, k, k, blocks.long()),
           lambda: dl.diffuser_selected_attention(q, k, k, blocks[:, :1]), lambda: dl.diffuser_selected_attention(q, k, k, blocks, out=q),
           lambda: dl.diffuser_selected_attention(q, k, k, blocks, lse=lse.double()),
           lambda: dl.diffuser_selected_attention(q, k.float(), k, blocks), lambda: dl.diffuser_selected_attention(q.cpu(), k, k, blocks),
           lambda: dl.diffuser_selected_attention(q, k, k, blocks, stream=torch.cuda.Stream(), lengths=i32.cpu()),
           lambda: dl.diffuser_selected_attention_backward(q, k, k.clone(), blocks, out, lse, out[:, :2]),
           lambda: dl.diffuser_selected_attention_backward(q, k, k.clone(), blocks, out, lse, out, dQ=out),
           lambda: dl.diffuser_selected_attention_backward(q, k, k.clone(), blocks, out, lse, out.clone(),
                                                           workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for x, call in enumerate(bad):
        with pytest.raises((dl.DiffuserError, ValueError, TypeError)):
            call()
            pytest.fail(f"call {x} was accepted")
    assert dl.diffuser_launch_count()[0] == before
    assert dl.diffuser_projection_status() == 0


def test_nothing_to_do(dl):
    """No queries, no sequences, no keys."""
    z = lambda *s: torch.zeros(s, dtype=BF, device="cuda")
    freq, _ = dl.diffuser_rope_frequencies()
    assert dl.diffuser_rope(z(1, 2, 0, 64), z(1, 1, 0, 64), freq)[0].shape == (1, 2, 0, 64)
    assert dl.diffuser_block_means(z(0, 1, 100, 64)).shape == (0, 1, 2, 64)
    assert dl.diffuser_block_means(z(1, 1, 0, 64)).shape == (1, 1, 0, 64)
    blocks = dl.diffuser_select_blocks(z(2, 2, 3, 64), z(2, 1, 0, 64), 4, keys=0)
    assert (blocks == -1).all()
    out, lse = dl.diffuser_selected_attention(z(2, 2, 3, 64) + 1, z(2, 1, 0, 64), z(2, 1, 0, 64), blocks, save_lse=True)
    assert not out.any() and (lse == -math.inf).all()
    for shape in ((2, 2, 0, 64), (0, 2, 3, 64)):
        q, k = z(*shape), z(shape[0], 1, 100, 64) + 1
        blocks = dl.diffuser_select_blocks(q, dl.diffuser_block_means(k), 2, keys=100)
        out, lse = dl.diffuser_selected_attention(q, k, k, blocks, save_lse=True)
        dq, dk, dv = dl.diffuser_selected_attention_backward(q, k, k.clone(), blocks, out, lse, q.clone(),
                                                             dK=torch.full_like(k, 7), dV=torch.full_like(k, 7))
        assert dq.shape == shape and not dk.any() and not dv.any()
    # queries that list nothing
    q, k = rand(70, 1, 2, 300, 64), rand(71, 1, 1, 300, 64)
    none = torch.full((1, 1, 300, 40), -1, dtype=torch.int32, device="cuda")
    out, lse = dl.diffuser_selected_attention(q, k, k, none, save_lse=True)
    grads = dl.diffuser_selected_attention_backward(q, k, k.clone(), none, out, lse, q.clone())
    assert not out.any() and (lse == -math.inf).all() and not any(g.any() for g in grads)


def test_status_is_clear(dl):
    torch.cuda.synchronize()
    assert dl.diffuser_projection_status() == 0


@pytest.mark.parametrize("n", [5, 400])
def test_scores_that_are_not_numbers(dl, n):
    """NaN in a query's row, or in a key that a row sees, is NaN in that row's result and log-sum, whether
    queries are few or many; rows that list no such block are what they were."""
    Hq, Hk, top = 8, 4, 8
    q, k, v = rand(1, 2, Hq, n, 64), rand(2, 2, Hk, 640, 64), rand(3, 2, Hk, 640, 64)
    blocks = torch.arange(top, dtype=torch.int32, device="cuda").expand(2, Hk, n, top).contiguous()
    blocks[:, :, 1] += 1                                     # row 1 lists all but block 0
    how = dict(causal=False, save_lse=True)
    out, lse = dl.diffuser_selected_attention(q, k, v, blocks, **how)
    bad = q.clone()
    bad[0, 3, 2, 5] = math.nan
    got, sums = dl.diffuser_selected_attention(bad, k, v, blocks, **how)
    hit = torch.zeros(2, Hq, n, dtype=torch.bool, device="cuda")
    hit[0, 3, 2] = True
    assert got[hit].isnan().all() and sums[hit].isnan().all()
    assert torch.equal(got[~hit], out[~hit]) and torch.equal(sums[~hit], lse[~hit])
    bad = k.clone()
    bad[1, 1, :64] = math.nan                                # all keys of a block of heads 2 and 3
    got, sums = dl.diffuser_selected_attention(q, bad, v, blocks, **how)
    hit = torch.zeros_like(hit)
    hit[1, 2:4] = True
    hit[:, :, 1] = False
    assert got[hit].isnan().all() and sums[hit].isnan().all()
    assert torch.equal(got[~hit], out[~hit]) and torch.equal(sums[~hit], lse[~hit])
