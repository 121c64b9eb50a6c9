"""The rotation alone and the attention over chosen key blocks, from their definitions, in 64
bits on the CPU."""
import math

import torch

BLOCK = 64


def rope(x, freq, magnitude, interleaved, pos):
    """x [B][H][n][64], pos int64 [B][n]."""
    r = 2 * len(freq)
    a = pos.double()[:, None, :, None] * torch.tensor(list(freq), dtype=torch.float64)
    z = torch.polar(torch.full_like(a, magnitude), a)
    head, rest = x[..., :r].double(), x[..., r:].double()
    if interleaved:
        head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (r // 2, 2)).contiguous()) * z).flatten(-2)
    else:
        w = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * z
        head = torch.cat((w.real, w.imag), -1)
    return torch.cat((head, rest), -1)


def limits(n, m, causal, length, start):
    """How many of the first keys each query of a sequence sees."""
    first = length - n if start is None else start
    out = []
    for i in range(n):
        p = first + i
        out.append(0 if p < 0 or p >= length else (p + 1 if causal else length))
    return out


def _sequences(B, n, m, lengths, starts):
    for b in range(B):
        length = m if lengths is None else min(max(int(lengths[b]), 0), m)
        yield b, length, None if starts is None else int(starts[b])


def means(K, lengths, old, recent=0):
    out = old.double().clone()
    B, _, m, _ = K.shape
    for b, length, _ in _sequences(B, 1, m, lengths, None):
        first = max(0, length - recent) // BLOCK if recent else 0
        for c in range(first, -(-length // BLOCK)):
            out[b, :, c] = K[b, :, c * BLOCK:min(length, (c + 1) * BLOCK)].double().sum(1) / (min(length, (c + 1) * BLOCK) - c * BLOCK)
    return out


def select(Q, mean, top, m, sink, local, causal, lengths, starts):
    B, Hq, n, _ = Q.shape
    Hk, nb = mean.shape[1:3]
    out = torch.full((B, Hk, n, top), -1, dtype=torch.int32)
    c = torch.arange(nb)
    for b, length, start in _sequences(B, n, m, lengths, starts):
        first = length - n if start is None else start
        count = -(-torch.tensor(limits(n, m, causal, length, start)) // BLOCK)     # blocks that each query sees
        home = torch.div(first + torch.arange(n), BLOCK, rounding_mode="floor")[:, None]
        forced = (c < sink) | ((c - home).abs() < local)
        most = max(1, int(count.max())) if n else 1
        for h in range(Hk):
            score = torch.zeros((n, nb), dtype=torch.float64)
            q, used = Q[b, h * (Hq // Hk):(h + 1) * (Hq // Hk)].double().transpose(0, 1), mean[b, h, :most].double()
            # (others are not read.)  The first two features by themselves: where they are large and cancel, a sum
            # that went on from them would lose 2^-33 of the others, and equal one score in 1e5 with another
            for part in (slice(0, 2), slice(2, 64)):
                score[:, :most] += q[..., part].flatten(1) @ used[:, part].repeat(1, Hq // Hk).T
            score = torch.where(score != score, -math.inf, score)
            rank = torch.sort(score, dim=1, descending=True, stable=True).indices      # equals by rising index
            group = torch.where(c[None] >= count[:, None], 2, torch.where(forced, 0, 1))
            rank = rank.gather(1, torch.sort(group.gather(1, rank), dim=1, stable=True).indices)[:, :top]
            taken = torch.where(torch.arange(rank.shape[1])[None] < count[:, None], rank, nb)
            taken = torch.sort(taken, dim=1).values
            out[b, h, :, :taken.shape[1]] = torch.where(taken < nb, taken, -1).to(torch.int32)
    return out


def mask(blocks, n, m, causal, lengths, starts):
    """Keys that each query sees, bool [B][Hk][n][m]."""
    B, Hk, _, top = blocks.shape
    out = torch.zeros((B, Hk, n, m), dtype=torch.bool)
    for b, length, start in _sequences(B, n, m, lengths, starts):
        lim = limits(n, m, causal, length, start)
        for h in range(Hk):
            for i in range(n):
                before = -1
                for c in blocks[b, h, i].tolist():
                    if c > before:
                        out[b, h, i, c * BLOCK:(c + 1) * BLOCK] = True
                    before = max(before, c)
                out[b, h, i, lim[i]:] = False
    return out


def attend(Q, K, V, seen):
    """out, lse, and sum_j p_ij |v_j|, the measure of out's roundings."""
    B, Hq, n, _ = Q.shape
    G = Hq // K.shape[1]
    on = seen.repeat_interleave(G, 1)
    k = torch.where(seen.any(2)[..., None], K.double(), 0.0).repeat_interleave(G, 1)     # (a key that no query sees is not read)
    v = torch.where(seen.any(2)[..., None], V.double(), 0.0).repeat_interleave(G, 1)
    x = (Q.double() @ k.mT / 8).masked_fill(~on, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse > -math.inf, lse, 0.0)[..., None])
    return p @ v, lse, p @ v.abs()


def gradients(Q, K, V, D, seen):
    """dQ, dK, dV by the formula, and for each the measures of its roundings: the sums of the
    absolute terms with dS (or P), and those with what dout.out's and dout.v's roundings make of dS."""
    B, Hq, n, _ = Q.shape
    Hk = K.shape[1]
    G = Hq // Hk
    on = seen.repeat_interleave(G, 1)
    used = seen.any(2)[..., None]
    k, v = (torch.where(used, x.double(), 0.0).repeat_interleave(G, 1) for x in (K, V))
    q, d = Q.double(), D.double()
    x = (q @ k.mT / 8).masked_fill(~on, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse > -math.inf, lse, 0.0)[..., None])
    out = p @ v
    dp = d @ v.mT
    ds = p * (dp - (d * out).sum(-1, keepdim=True)) / 8
    coarse = p * (d.abs() * out.abs()).sum(-1, keepdim=True) / 8     # times u: dout.out of the rounded out
    fine = p * (d.abs() @ v.abs().mT) / 8                            # times 2^-16: dout.v in fp32

    def heads(y):
        return y.unflatten(1, (Hk, G)).sum(2)

    return ((ds @ k, heads(ds.mT @ q), heads(p.mT @ d)),
            (ds.abs() @ k.abs(), heads(ds.abs().mT @ q.abs()), heads(p.mT @ d.abs())),
            (coarse @ k.abs(), heads(coarse.mT @ q.abs()), 0.0),
            (fine @ k.abs(), heads(fine.mT @ q.abs()), 0.0))
