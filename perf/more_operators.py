"""Attention over key blocks that a cheap score chooses for each query, and what it stands
on, timed and compared: rotary positions scaled for long contexts, the means of key blocks,
the choice of blocks, the attention over them and its backward pass.

`run` computes them in plain torch operations, or, with `own` set, by the calls a user makes
of the library's binding.
"""
import math

import torch

own = False

HEAD = 64                       # head width of the library
BLOCK = 64                      # keys of a block
THETA, ORIGINAL = 10000.0, 4096     # rotation base; the context that the scalings stretch
SCALINGS = ("none", "linear", "ntk", "yarn")


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token for each of 16 sequences of a server, each at a position of its own (up to
        # a million), 16 query and 4 key heads, YaRN frequencies: launch latency
        _rope("rope_decode_b16", B=16, Hq=16, Hk=4, n=1, dtype="bf16", scaling="yarn", far=True),
        # the long workload's queries and keys (16 heads x 16384 tokens) at four times the trained context
        _rope("rope_long", B=1, Hq=16, Hk=16, n=16384, dtype="bf16", scaling="yarn"),
        # fp32 I/O, an odd length, half of the width turned in neighbouring pairs, gradients
        _rope("rope_fp32_odd_backward", B=3, Hq=12, Hk=4, n=1021, dtype="fp32", scaling="ntk", rot=32,
              interleaved=True, far=True, backward=True),
        # a server's step appended one key to each of 16 caches: the mean of the block it fell into
        _means("means_append_b16", B=16, Hk=4, m=65536, recent=1, ragged=True),
        # the long workload's keys, a prompt or a training step
        _means("means_long", B=1, Hk=16, m=16384),
        # a server's step: blocks for one token of 16 sequences with up to 65536 cached keys
        _select("select_decode_b16", B=16, Hq=16, Hk=4, n=1, m=65536, top=16, sink=1, local=2, ragged=True),
        # the long workload: blocks for every token of every head
        _select("select_long", B=1, Hq=16, Hk=16, n=16384, m=16384, top=16, sink=1, local=2),
        # the same server's attention over its chosen blocks
        _attend("attend_decode_b16", B=16, Hq=16, Hk=4, n=1, m=65536, top=16, sink=1, local=2, ragged=True),
        # the text workload (2 x 12 heads x 4096 tokens), bidirectional, log-sums kept for the backward
        _attend("attend_text", B=2, Hq=12, Hk=12, n=4096, m=4096, top=8, sink=1, local=1, causal=False, save=True),
        # the long workload, causal
        _attend("attend_long", B=1, Hq=16, Hk=16, n=16384, m=16384, top=16, sink=1, local=2),
        # training on a right-padded batch of odd length with three query heads to a key head
        _attend("attend_odd_backward", B=3, Hq=12, Hk=4, n=1021, m=1021, top=6, sink=1, local=2, ragged=True,
                backward=True),
        # training on the long workload: the largest case
        _attend("attend_long_backward", B=1, Hq=16, Hk=16, n=16384, m=16384, top=16, sink=1, local=2, backward=True),
    ]


def _named(name, c):
    return dict(c, name=name) if name else c


def _rope(name, B, Hq, Hk, n, dtype, scaling, rot=HEAD, interleaved=False, far=False, backward=False):
    return _named(name, dict(op="rope", B=B, Hq=Hq, Hk=Hk, n=n, dtype=dtype, scaling=scaling, rot=rot,
                             interleaved=interleaved, far=far, backward=backward))


def _means(name, B, Hk, m, recent=0, ragged=False):
    return _named(name, dict(op="means", B=B, Hk=Hk, m=m, recent=recent, ragged=ragged))


def _select(name, B, Hq, Hk, n, m, top, sink, local, causal=True, ragged=False):
    return _named(name, dict(op="select", B=B, Hq=Hq, Hk=Hk, n=n, m=m, top=top, sink=sink, local=local,
                             causal=causal, ragged=ragged))


def _attend(name, B, Hq, Hk, n, m, top, sink, local, causal=True, ragged=False, save=False, backward=False):
    return _named(name, dict(op="attend", B=B, Hq=Hq, Hk=Hk, n=n, m=m, top=top, sink=sink, local=local,
                             causal=causal, ragged=ragged, save=save, backward=backward))


MOST_ROWS = 2 * 16 * 16384                 # of the largest listed rotation
MOST_SCORES = 16 * 16384 * 256             # of the largest listed choice
MOST_PAIRS = 16 * 16384 * 16               # (query row, block) pairs of the largest listed attention
MOST_CACHE = 16 * 4 * 65536                # keys of the largest listed cache


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "means", "select", "attend", "attend"))
    while True:
        B, Hk = _log(rng, 1, 32), rng.randint(1, 16)
        if op == "rope":
            c = _rope(None, B=B, Hq=rng.randint(1, 16), Hk=Hk, n=_log(rng, 1, 16384), dtype=rng.choice(("bf16", "fp32")),
                      scaling=rng.choice(SCALINGS), rot=16 * rng.randint(1, 4), interleaved=rng.random() < 0.5,
                      far=rng.random() < 0.5, backward=rng.random() < 0.5)
            if B * (c["Hq"] + Hk) * c["n"] <= MOST_ROWS:
                return c
            continue
        if op == "means":
            c = _means(None, B=B, Hk=Hk, m=_log(rng, 1, 65536), recent=rng.choice((0, 1, rng.randint(1, 200))),
                       ragged=rng.random() < 0.5)
            if B * Hk * c["m"] <= MOST_CACHE:
                return c
            continue
        Hq = Hk * rng.randint(1, max(1, 16 // Hk))
        if rng.random() < 0.4:             # a step of a few tokens on a cache
            n, m = _log(rng, 1, 8), _log(rng, 8, 65536)
        else:
            n = m = _log(rng, 1, 16384)
        causal, sink, local = rng.random() < 0.7, rng.randint(0, 2), rng.randint(0, 2)
        forced = sink + (local if causal else max(0, 2 * local - 1))
        how = dict(B=B, Hq=Hq, Hk=Hk, n=n, m=m, top=max(1, forced, _log(rng, 1, 32)), sink=sink, local=local,
                   causal=causal, ragged=rng.random() < 0.5)
        if B * Hk * m > MOST_CACHE:
            continue
        if op == "select":
            if B * Hq * n * _blocks(m) <= MOST_SCORES:
                return _select(None, **how)
            continue
        backward = rng.random() < 0.5
        if B * Hq * n * min(how["top"], _blocks(m)) <= MOST_PAIRS:
            return _attend(None, backward=backward, save=not backward and rng.random() < 0.5, **how)


def _blocks(m):
    return -(-m // BLOCK)


def _listed_blocks(c):
    """Blocks that a query lists, on average, where nothing is padded."""
    nb = _blocks(c["m"])
    top = min(c["top"], nb)
    if not c["causal"] or c["n"] < c["m"]:
        return float(top)
    return top - top * (top - 1) / (2 * nb)        # the first blocks' queries see fewer


def work(case):
    if case["op"] == "rope":
        e = case["B"] * (case["Hq"] + case["Hk"]) * case["n"] * HEAD
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * e * size + (8 * case["B"] * case["n"] if case["far"] else 0),
                "flops": 6 * e * case["rot"] // HEAD}
    fill = 0.625 if case["ragged"] else 1.0        # lengths are spread over a quarter to all of m
    m, units = case["m"] * fill, case["B"] * case["Hk"]
    if case["op"] == "means":
        keys = units * (min(m, case["recent"] + BLOCK / 2) if case["recent"] else m)
        return {"bytes": int(2 * HEAD * keys * (1 + 1 / BLOCK)), "flops": int(HEAD * keys)}
    n = case["n"] * (fill if case["n"] == case["m"] else 1)
    rows, nb = case["B"] * case["Hq"] * n, _blocks(m)
    if case["op"] == "select":
        scores = rows * (nb if not case["causal"] or case["n"] < case["m"] else nb / 2)
        return {"bytes": int(2 * HEAD * (rows + units * nb) + 4 * case["B"] * case["Hk"] * n * case["top"]),
                "flops": int(2 * HEAD * scores)}
    pairs = rows * _listed_blocks(case)
    keys = min(units * m, case["B"] * case["Hk"] * n * _listed_blocks(case) * BLOCK)
    index = 4 * case["B"] * case["Hk"] * n * case["top"]
    if case["backward"]:                           # Q, out, dOut, dQ; K, V, dK, dV; log-sums
        return {"bytes": int(2 * HEAD * (4 * rows + 4 * keys) + 4 * rows + index), "flops": int(10 * HEAD * BLOCK * pairs)}
    return {"bytes": int(2 * HEAD * (2 * rows + 2 * keys) + (4 * rows if case["save"] else 0) + index),
            "flops": int(4 * HEAD * BLOCK * pairs)}


# ------------------------------------------------------------------ the inputs
def _plan(case):
    """Frequencies (radians per position) and magnitude of a scaling, in 64 bits."""
    r, kind = case["rot"], case["scaling"]
    f = [THETA ** (-2 * i / r) for i in range(r // 2)]
    s = 4.0                                        # four times the trained context
    if kind == "linear":
        return [x / s for x in f], 1.0
    if kind == "ntk":
        base = THETA * s ** (r / (r - 2))
        return [base ** (-2 * i / r) for i in range(r // 2)], 1.0
    if kind == "yarn":
        keep = [min(1.0, max(0.0, (ORIGINAL * x / (2 * math.pi) - 1) / (32 - 1))) for x in f]
        return [x * (g + (1 - g) / s) for x, g in zip(f, keep)], 1 + 0.1 * math.log(s)
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    s, B, Hk = {"case": case}, case["B"], case["Hk"]
    if case["op"] == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["q"], s["k"] = normal(B, case["Hq"], case["n"], HEAD, dtype=dt), normal(B, Hk, case["n"], HEAD, dtype=dt)
        s["pos"] = None
        if case["far"]:                            # each sequence runs on from a position of its own
            first = torch.randint(0, 1 << 20, (B, 1), generator=g, device="cuda")
            s["pos"] = first + torch.arange(case["n"], device="cuda")
        s["freq"], s["magnitude"] = _plan(case)
        if own:                                    # a program makes its frequencies once
            from sparse_long_sequence_gb300 import binding as dl
            s["freq"], s["magnitude"] = dl.diffuser_rope_frequencies(
                case["rot"], theta=THETA, scaling=getattr(dl, "DIFFUSER_ROPE_" + case["scaling"].upper()), factor=4.0,
                original_length=ORIGINAL)
        return s

    m, nb = case["m"], _blocks(case["m"])
    s["len"] = s["start"] = None
    if case["ragged"]:
        low = max(1, m // 4, min(case.get("n", 1), m))
        if case.get("n") == m:
            low = max(1, m // 4)
            s["start"] = torch.zeros(B, dtype=torch.int32, device="cuda")      # padded on the right
        s["len"] = torch.randint(low, m + 1, (B,), generator=g, device="cuda").to(torch.int32)
    # texts stay on a topic for a block or so: keys lean to their block's topic, and a query to
    # one topic of 32 of its own
    topics = torch.randn((Hk, 32, HEAD), generator=g, device="cuda")
    of = torch.randint(0, 32, (B, 1, nb), generator=g, device="cuda").expand(B, Hk, nb)
    lean = topics[torch.arange(Hk, device="cuda")[None, :, None], of]
    k = torch.randn((B, Hk, m, HEAD), generator=g, device="cuda")
    s["k"] = k.mul_(0.8).add_(lean.repeat_interleave(BLOCK, 2)[:, :, :m], alpha=0.6).bfloat16()
    del k
    if case["op"] == "means":
        s["means"] = torch.zeros((B, Hk, nb, HEAD), dtype=torch.bfloat16, device="cuda")
        if case["recent"]:                         # what the server has from before the step
            length = s["len"] if s["len"] is not None else torch.full((B,), m, device="cuda", dtype=torch.int32)
            _write_means(s["k"], (length - case["recent"]).clamp(min=0), 0, s["means"])
        return s
    n, G = case["n"], case["Hq"] // Hk
    wants = torch.randint(0, 32, (B, Hk, n), generator=g, device="cuda")
    q = topics[torch.arange(Hk, device="cuda")[None, :, None], wants][:, :, None] * 0.6
    s["q"] = (q + torch.randn((B, Hk, G, n, HEAD), generator=g, device="cuda") * 0.8).view(B, Hk * G, n, HEAD).bfloat16()
    means = torch.zeros((B, Hk, nb, HEAD), dtype=torch.bfloat16, device="cuda")
    _write_means(s["k"], s["len"], 0, means)
    if case["op"] == "select":
        s["means"] = means
        return s
    s["v"] = normal(B, Hk, m, HEAD)
    s["blocks"] = _choose(case, s["q"], means, s["len"], s["start"])
    if case["backward"]:                           # what the forward has kept
        s["out"], s["lse"] = _attend_plain(s)
        s["dout"] = normal(*s["q"].shape)
    return s


# ------------------------------------------------------------------ plain forms
def _rope_plain(s):
    c = s["case"]
    pos = s["pos"] if s["pos"] is not None else torch.arange(c["n"], device="cuda")[None]
    freq, mag = _plan(c)                           # angles in 64 bits: positions are far
    a = pos[:, None, :, None].double() * torch.tensor(freq, dtype=torch.float64, device="cuda")
    cos, sin = (torch.cos(a) * mag).float(), (torch.sin(a) * (-mag if c["backward"] else mag)).float()
    out, r = [], c["rot"]
    for x in (s["q"], s["k"]):
        f = x.float()
        if c["interleaved"]:
            u, v = f[..., 0:r:2], f[..., 1:r:2]
            turned = torch.stack((u * cos - v * sin, u * sin + v * cos), -1).flatten(-2)
        else:
            u, v = f[..., :r // 2], f[..., r // 2:r]
            turned = torch.cat((u * cos - v * sin, u * sin + v * cos), -1)
        out.append(torch.cat((turned, f[..., r:]), -1).to(x.dtype))
    return out


def _write_means(k, length, recent, means):
    """The means of the blocks below each length (recent: of those that hold the last tokens)."""
    B, Hk, m, _ = k.shape
    nb = _blocks(m)
    if length is None:
        length = torch.full((B,), m, device=k.device, dtype=torch.int32)
    first = ((length - recent).clamp(min=0) // BLOCK if recent else torch.zeros_like(length)).long()
    count = -(-length.long() // BLOCK) - first     # blocks to do of each sequence
    most = min(nb, -(-recent // BLOCK) + 1) if recent else nb
    c = first[:, None] + torch.arange(most, device=k.device)
    todo = torch.arange(most, device=k.device)[None] < count[:, None]
    c = torch.where(todo, c, torch.zeros_like(c))
    at = c[:, :, None] * BLOCK + torch.arange(BLOCK, device=k.device)
    live = at < length[:, None, None]
    rows = torch.arange(B, device=k.device)[:, None, None]
    for h in range(Hk):                            # a head at a time: long caches in 32 bits
        x = torch.where(live[..., None], k[rows, h, at.clamp(max=m - 1)].float(), torch.zeros((), device=k.device))
        mean = x.sum(2) / live.sum(2).clamp(min=1)[..., None]
        old = means[rows[..., 0], h, c]
        new = torch.where(todo[..., None], mean.to(means.dtype), old)
        if recent:                                 # (block by block: places left over stand at block 0)
            for j in range(most):
                means[rows[:, 0, 0], h, c[:, j]] = torch.where(todo[:, j, None], new[:, j],
                                                               means[rows[:, 0, 0], h, c[:, j]])
        else:
            means[:, h] = torch.where(todo[..., None], new, means[:, h])
    return means


def _places(case, length, start, device):
    """Position of each query [B][n], and the lengths [B]."""
    B, n, m = case["B"], case["n"], case["m"]
    if length is None:
        length = torch.full((B,), m, device=device)
    first = (length - n) if start is None else start
    return first.long()[:, None] + torch.arange(n, device=device), length.long()


def _choose(case, q, means, length, start):
    """Blocks [B][Hk][n][top], ascending, -1 behind them; scores in 64 bits (near ties decide)."""
    B, Hq, n, _ = q.shape
    Hk, nb, top = means.shape[1], means.shape[2], case["top"]
    pos, length = _places(case, length, start, q.device)
    score = torch.einsum("bhgnd,bhcd->bhnc", q.view(B, Hk, Hq // Hk, n, HEAD).double(), means.double())
    c = torch.arange(nb, device=q.device)
    seen = (c * BLOCK < length[:, None])[:, None] & ((pos >= 0) & (pos < length[:, None]))[..., None]
    if case["causal"]:
        seen = seen & (c * BLOCK <= pos[..., None])
    own_block = torch.div(pos, BLOCK, rounding_mode="floor")[..., None]
    forced = (c < case["sink"]) | ((c - own_block).abs() < case["local"])
    score = torch.where(forced[:, None], torch.full_like(score[:1, :1, :1], math.inf), score)
    score = torch.where(seen[:, None], score, torch.full_like(score[:1, :1, :1], -math.inf))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    count = seen.sum(-1)[:, None, :, None]
    rank = torch.arange(order.shape[-1], device=q.device)
    order = torch.where(rank < count, order, torch.full_like(order, nb))
    order = torch.sort(order, dim=-1).values
    out = torch.full((B, Hk, n, top), -1, dtype=torch.int32, device=q.device)
    out[..., :order.shape[-1]] = torch.where(order < nb, order, torch.full_like(order, -1)).to(torch.int32)
    return out


def _gathered(s):
    """Chunks of (batch, key head, query) rows: their slice, the rows of K and V that they
    list [rows][keys], and which of those they see."""
    c, k = s["case"], s["k"]
    B, Hk, n, top = s["blocks"].shape
    m = k.shape[2]
    pos, length = _places(c, s["len"], s["start"], k.device)
    blocks = s["blocks"].view(-1, top)
    unit = torch.arange(B * Hk, device=k.device).repeat_interleave(n)
    pos, length = pos[:, None].expand(B, Hk, n).reshape(-1), length[:, None, None].expand(B, Hk, n).reshape(-1)
    step = max(1, (1 << 22) // (top * BLOCK))
    for a in range(0, blocks.shape[0], step):
        e = slice(a, a + step)
        key = blocks[e].long()[..., None] * BLOCK + torch.arange(BLOCK, device=k.device)
        p, l = pos[e, None, None], length[e, None, None]
        seen = (blocks[e] >= 0)[..., None] & (key < l) & (p >= 0) & (p < l)
        if c["causal"]:
            seen = seen & (key <= p)
        row = unit[e, None, None] * m + key.clamp(0, m - 1)
        yield e, row.flatten(1), seen.flatten(1)


def _by_unit(c, x):
    """[B][Hq][n][w] as [B Hk n][G][w]."""
    return x.view(c["B"], c["Hk"], c["Hq"] // c["Hk"], c["n"], -1).transpose(2, 3).flatten(0, 2)


def _by_head(c, x):
    return x.view(c["B"], c["Hk"], c["n"], c["Hq"] // c["Hk"], -1).transpose(2, 3).reshape(c["B"], c["Hq"], c["n"], -1)


def _attend_plain(s):
    c = s["case"]
    q, k, v = _by_unit(c, s["q"]), s["k"].view(-1, HEAD), s["v"].view(-1, HEAD)
    out = torch.zeros(q.shape, device=q.device)
    lse = torch.zeros(q.shape[:2], device=q.device)
    for e, row, seen in _gathered(s):
        x = q[e].float() @ k[row].float().mT * HEAD ** -0.5
        x = torch.where(seen[:, None], x, torch.full_like(x[:1, :1, :1], -math.inf))
        top = x.max(-1, keepdim=True).values
        top = torch.where(top > -math.inf, top, torch.zeros_like(top))
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        out[e] = p @ v[row].float() / torch.where(total > 0, total, torch.ones_like(total))
        lse[e] = (top + torch.log(total))[..., 0]
    return _by_head(c, out).bfloat16(), _by_head(c, lse[..., None])[..., 0].contiguous()


def _attend_plain_backward(s):
    c = s["case"]
    q, k, v = _by_unit(c, s["q"]), s["k"].view(-1, HEAD), s["v"].view(-1, HEAD)
    lse, out, dout = _by_unit(c, s["lse"][..., None]), _by_unit(c, s["out"]), _by_unit(c, s["dout"])
    dq = torch.zeros(q.shape, device=q.device)
    dk, dv = torch.zeros(k.shape, device=q.device), torch.zeros(v.shape, device=q.device)
    for e, row, seen in _gathered(s):
        qe, ke, ve, de = q[e].float(), k[row].float(), v[row].float(), dout[e].float()
        l = torch.where(lse[e] > -math.inf, lse[e], torch.zeros_like(lse[e]))
        p = torch.where(seen[:, None], torch.exp(qe @ ke.mT * HEAD ** -0.5 - l), torch.zeros_like(ke[:1, :1, :1]))
        dp = de @ ve.mT
        ds = p * (dp - (de * out[e].float()).sum(-1, keepdim=True)) * HEAD ** -0.5
        dq[e] = ds @ ke
        dk.index_add_(0, row.flatten(), (ds.mT @ qe).flatten(0, 1))
        dv.index_add_(0, row.flatten(), (p.mT @ de).flatten(0, 1))
    return [_by_head(c, dq).bfloat16(), dk.view(s["k"].shape).bfloat16(), dv.view(s["v"].shape).bfloat16()]


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    from sparse_long_sequence_gb300 import binding as dl
    c = s["case"]
    if c["op"] == "rope":
        call = dl.diffuser_rope_backward if c["backward"] else dl.diffuser_rope
        return list(call(s["q"], s["k"], s["freq"], magnitude=s["magnitude"], interleaved=c["interleaved"],
                         positions=s["pos"]))
    if c["op"] == "means":
        return [dl.diffuser_block_means(s["k"], lengths=s["len"], recent=c["recent"], means=s["means"])]
    if c["op"] == "select":
        return [dl.diffuser_select_blocks(s["q"], s["means"], c["top"], keys=c["m"], sink_blocks=c["sink"],
                                          local_blocks=c["local"], causal=c["causal"], lengths=s["len"],
                                          starts=s["start"])]
    how = dict(causal=c["causal"], lengths=s["len"], starts=s["start"])
    if c["backward"]:                              # (the call takes contiguous tensors; the plain forward may keep a view)
        return list(dl.diffuser_selected_attention_backward(s["q"], s["k"], s["v"], s["blocks"], s["out"].contiguous(),
                                                            s["lse"], s["dout"], **how))
    out = dl.diffuser_selected_attention(s["q"], s["k"], s["v"], s["blocks"], save_lse=c["save"], **how)
    return list(out) if c["save"] else [out]


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "rope":
        return _rope_plain(state)
    if c["op"] == "means":
        return [_write_means(state["k"], state["len"], c["recent"], state["means"])]
    if c["op"] == "select":
        return [_choose(c, state["q"], state["means"], state["len"], state["start"])]
    if c["backward"]:
        return _attend_plain_backward(state)
    out, lse = _attend_plain(state)
    return [out, lse] if c["save"] else [out]


# ------------------------------------------------------------------ in 64 bits
def _exact_rope(c, s):
    """Pairs as complex numbers, each times m exp(i angle); the backward as its conjugate."""
    freq, mag = _plan(c)
    pos = s["pos"] if s["pos"] is not None else torch.arange(c["n"], device="cuda").expand(c["B"], -1)
    ang = pos.double()[:, None, :, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    w = torch.polar(torch.full_like(ang, mag), -ang if c["backward"] else ang)
    out, r = [], c["rot"]
    for x in (s["q"].double(), s["k"].double()):
        head, rest = x[..., :r], x[..., r:]
        if c["interleaved"]:
            z = torch.view_as_complex(head.unflatten(-1, (r // 2, 2)).contiguous()) * w
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * w
            head = torch.cat((z.real, z.imag), -1)
        out.append(torch.cat((head, rest), -1))
    return out


def _lengths(c, s):
    """Each sequence's length and its first query's position, as numbers."""
    length = s["len"].tolist() if s["len"] is not None else [c["m"]] * c["B"]
    start = s["start"].tolist() if s["start"] is not None else [x - c["n"] for x in length]
    return length, start


def _exact_means(c, s):
    means = s["means"].double()
    for b, length in enumerate(_lengths(dict(c, n=1), s)[0]):
        first = max(0, length - c["recent"]) // BLOCK if c["recent"] else 0
        for i in range(first, _blocks(length)):
            means[b, :, i] = s["k"][b, :, i * BLOCK:min(length, (i + 1) * BLOCK)].double().mean(1)
    return [means]


def _exact_select(c, s):
    """By counting, for each block, how many come before it."""
    G, nb = c["Hq"] // c["Hk"], _blocks(c["m"])
    out = torch.full((c["B"], c["Hk"], c["n"], c["top"]), -1, dtype=torch.int32, device="cuda")
    idx = torch.arange(nb, device="cuda")
    length, start = _lengths(c, s)
    step = max(1, (1 << 25) // (nb * nb))
    for b in range(c["B"]):
        for h in range(c["Hk"]):
            total = s["q"][b, h * G:(h + 1) * G].double().sum(0)
            mean = s["means"][b, h].double()
            for a in range(0, c["n"], step):
                p = start[b] + torch.arange(a, min(c["n"], a + step), device="cuda")[:, None]
                x = total[a:a + step] @ mean.T
                home = torch.div(p, BLOCK, rounding_mode="floor")
                x = x.masked_fill((idx < c["sink"]) | ((idx - home).abs() < c["local"]), math.inf)
                off = (p < 0) | (p >= length[b]) | (idx * BLOCK >= length[b])
                if c["causal"]:
                    off = off | (idx * BLOCK > p)
                x = x.masked_fill(off, -math.inf)
                before = (x[:, None] > x[..., None]) | ((x[:, None] == x[..., None]) & (idx < idx[:, None]))
                take = (before.sum(-1) < c["top"]) & ~off
                place = take.cumsum(1) - 1
                r, col = take.nonzero(as_tuple=True)
                out[b, h, a + r, place[r, col]] = col.to(torch.int32)
    return [out]


def _exact_attend(c, s):
    """Dense over all keys, a few rows of a head at a time; gradients by automatic differentiation."""
    G, m, nb = c["Hq"] // c["Hk"], c["m"], _blocks(c["m"])
    length, start = _lengths(c, s)
    wide = {x: s[x].double() for x in ("q", "k", "v", "dout") if x in s}
    outs = [torch.zeros_like(wide[x]) for x in (("q", "k", "v") if c["backward"] else ("q",))]
    sums = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    idx = torch.arange(m, device="cuda")
    step = max(1, (1 << 27) // (m * G))
    for b in range(c["B"]):
        for h in range(c["Hk"]):
            heads = slice(h * G, (h + 1) * G)
            k, v = wide["k"][b, h], wide["v"][b, h]
            live = (idx < length[b])[:, None]
            k, v = torch.where(live, k, 0.0).requires_grad_(c["backward"]), torch.where(live, v, 0.0).requires_grad_(c["backward"])
            for a in range(0, c["n"], step):
                rows = slice(a, min(c["n"], a + step))
                q = wide["q"][b, heads, rows].clone().requires_grad_(c["backward"])
                chosen = s["blocks"][b, h, rows].long()
                on = torch.zeros((chosen.shape[0], nb + 1), dtype=torch.bool, device="cuda")
                on.scatter_(1, torch.where(chosen < 0, nb, chosen), True)
                p = start[b] + torch.arange(rows.start, rows.stop, device="cuda")[:, None]
                on = on[:, :nb].repeat_interleave(BLOCK, 1)[:, :m] & (idx < length[b]) & (p >= 0) & (p < length[b])
                if c["causal"]:
                    on = on & (idx <= p)
                some = on.any(1)
                x = torch.einsum("gnd,md->gnm", q, k).div(math.sqrt(HEAD)).masked_fill(~on, -math.inf)
                weight = torch.softmax(x[:, some], -1)
                y = torch.einsum("gnm,md->gnd", weight, v)
                if c["backward"]:
                    gq, gk, gv = torch.autograd.grad(y, (q, k, v), wide["dout"][b, heads, rows][:, some])
                    outs[0][b, heads, rows] = gq
                    outs[1][b, h] += gk
                    outs[2][b, h] += gv
                else:
                    at = some.nonzero()[:, 0] + a
                    outs[0][b, heads, at] = y
                    sums[b, heads, at] = torch.logsumexp(x[:, some], -1)
    return outs + [sums] if c.get("save") else outs


def exact(case, seed):
    if case["op"] == "attend":
        products = 7 if case["backward"] else 2
        if 2 * HEAD * products * case["B"] * case["Hq"] * case["n"] * case["m"] > 8e12:
            return None                            # over 20 seconds
    if case["op"] == "select" and case["B"] * case["Hk"] * case["n"] * _blocks(case["m"]) ** 2 > 6e10:
        return None
    if case["op"] == "means" and not case["recent"] and case["B"] * _blocks(case["m"]) > 20000:
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "means": _exact_means, "select": _exact_select,
            "attend": _exact_attend}[case["op"]](case, s)
