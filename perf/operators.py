"""The operators around the diffusion module that are timed and compared: the
per-head norms of queries and keys with the position rotation, the dense product
with its epilogue, and the gated feed-forward product, each forward and backward.

`run` computes them in plain fp32 torch operations, or, with `own` set, by the
calls a user makes of the library's binding.
"""
import math

import torch

own = False

HEAD = 64                       # head width of the library
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token for each of 16 sequences of a server, each at a position of its own
        # (up to a million), queries and keys of 16 heads: launch latency
        _qk("qk_decode_b16", B=16, Hq=16, Hk=16, n=1, dtype="bf16", far=True),
        # the text workload's queries and keys (2 x 12 heads x 4096 tokens), from position 0
        _qk("qk_text", B=2, Hq=12, Hk=12, n=4096, dtype="bf16"),
        # fp32 I/O, fewer key heads than query heads, an odd length, half of the width rotated
        # in neighbouring pairs, positions given per token (packed or left-padded batches)
        _qk("qk_fp32_odd", B=3, Hq=12, Hk=4, n=1021, dtype="fp32", rot=32, interleaved=True, far=True),
        # training on the long workload (16 heads x 16384 tokens): gradients of queries, keys
        # and both norm weights
        _qk("qk_long_backward", B=1, Hq=16, Hk=16, n=16384, dtype="bf16", backward=True),
        # a server's step of 4 tokens through a 1024 -> 4096 product with bias and gelu: the
        # weights are read once, nothing else matters
        _linear("linear_decode_t4", T=4, D=1024, F=4096, act="gelu", bias=True),
        # the text layer's output projection (8192 tokens, 768 -> 768) with bias and residual
        _linear("linear_text_residual", T=8192, D=768, F=768, act="none", bias=True, residual=True),
        # the long-range batch's feed-forward (32768 tokens, 512 -> 2048) in training: gelu, with
        # the pre-activations kept
        _linear("linear_lra_gelu_train", T=32768, D=512, F=2048, act="gelu_tanh", bias=True, save=True),
        # its backward at the long workload's width: gradients of input, weights and bias
        _linear("linear_long_backward", T=16384, D=1024, F=4096, act="gelu_tanh", bias=True, backward=True),
        # a server's step of 16 tokens through the gated product
        _gated("gated_decode_t16", T=16, D=1024, F=2816, act="silu"),
        # a ragged prompt at odd widths (no multiple of any tile)
        _gated("gated_ragged", T=777, D=520, F=1368, act="gelu_tanh"),
        # the text workload's feed-forward (8192 tokens, 768 -> 2048) in training
        _gated("gated_text_train", T=8192, D=768, F=2048, act="silu", save=True),
        # the long workload's, backward: the largest case
        _gated("gated_long_backward", T=16384, D=1024, F=2816, act="silu", backward=True),
    ]


def _qk(name, B, Hq, Hk, n, dtype, rot=HEAD, interleaved=False, far=False, backward=False):
    c = dict(op="qk", B=B, Hq=Hq, Hk=Hk, n=n, dtype=dtype, rot=rot, interleaved=interleaved, far=far,
             backward=backward)
    return dict(c, name=name) if name else c


def _linear(name, T, D, F, act, bias=False, residual=False, save=False, backward=False):
    c = dict(op="linear", T=T, D=D, F=F, act=act, bias=bias, residual=residual, save=save, backward=backward)
    return dict(c, name=name) if name else c


def _gated(name, T, D, F, act, save=False, backward=False):
    c = dict(op="gated", T=T, D=D, F=F, act=act, save=save, backward=backward)
    return dict(c, name=name) if name else c


MOST_FLOPS = 8 * 16384 * 1024 * 2816     # of the largest listed case
MOST_BYTES = 6 * 16 * 16384 * HEAD * 2   # of the largest listed norm-and-rotation


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("qk", "linear", "gated"))
    while True:
        if op == "qk":
            B, Hq, Hk = _log(rng, 1, 32), rng.randint(1, 16), rng.randint(1, 16)
            c = _qk(None, B=B, Hq=Hq, Hk=Hk, n=_log(rng, 1, 16384), dtype=rng.choice(("bf16", "fp32")),
                    rot=16 * rng.randint(1, 4), interleaved=rng.random() < 0.5, far=rng.random() < 0.5,
                    backward=rng.random() < 0.5)
        else:
            T, D, F = _log(rng, 1, 32768), 8 * _log(rng, 8, 256), 8 * _log(rng, 8, 512)
            backward = rng.random() < 0.5
            if op == "linear":
                c = _linear(None, T=T, D=D, F=F, act=rng.choice(ACTS), bias=rng.random() < 0.7,
                            residual=not backward and rng.random() < 0.5,
                            save=not backward and rng.random() < 0.5, backward=backward)
            else:
                c = _gated(None, T=T, D=D, F=F, act=rng.choice(ACTS[1:]),
                           save=not backward and rng.random() < 0.5, backward=backward)
        w = work(c)
        if w["flops"] <= MOST_FLOPS and (op != "qk" or w["bytes"] <= MOST_BYTES):
            return c


def work(case):
    if case["op"] == "qk":
        e = case["B"] * (case["Hq"] + case["Hk"]) * case["n"] * HEAD
        size = 2 if case["dtype"] == "bf16" else 4
        if case["backward"]:
            return {"bytes": 3 * e * size + 4 * HEAD * size, "flops": 18 * e}
        return {"bytes": 2 * e * size + 2 * HEAD * size, "flops": 8 * e}
    T, D, F = case["T"], case["D"], case["F"]
    if case["op"] == "linear":
        if case["backward"]:
            ins = T * D + F * D + T * F * (2 if case["act"] != "none" else 1)
            return {"bytes": 2 * (ins + T * D + F * D + (F if case["bias"] else 0)), "flops": 4 * T * D * F}
        extra = (F if case["bias"] else 0) + T * F * (int(case["residual"]) + int(case["save"]))
        return {"bytes": 2 * (T * D + F * D + T * F + extra), "flops": 2 * T * D * F}
    if case["backward"]:
        return {"bytes": 2 * (2 * T * D + 4 * F * D + 3 * T * F), "flops": 8 * T * D * F}
    return {"bytes": 2 * (T * D + 2 * F * D + T * F * (3 if case["save"] else 1)), "flops": 4 * T * D * F}


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, scale=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "qk":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        B, n = case["B"], case["n"]
        s["q"], s["k"] = normal(B, case["Hq"], n, HEAD, dtype=dt), normal(B, case["Hk"], n, HEAD, dtype=dt)
        s["wq"] = normal(HEAD, dtype=dt, scale=0.2, mean=1.0)
        s["wk"] = normal(HEAD, dtype=dt, scale=0.2, mean=1.0)
        # each sequence runs on from a position of its own, up to 2^20
        s["pos"] = None
        if case["far"]:
            first = torch.randint(0, 1 << 20, (B, 1), generator=g, device="cuda")
            s["pos"] = first + torch.arange(n, device="cuda")
        if case["backward"]:
            s["dq"], s["dk"] = normal(*s["q"].shape, dtype=dt), normal(*s["k"].shape, dtype=dt)
        return s
    T, D, F = case["T"], case["D"], case["F"]
    rows = F if case["op"] == "linear" else 2 * F
    s["x"] = normal(T, D)
    s["w"] = normal(rows, D, scale=D ** -0.5)
    s["bias"] = normal(F, scale=0.1) if case.get("bias") else None
    s["res"] = normal(T, F) if case.get("residual") else None
    if case["backward"]:
        s["dy"] = normal(T, F)
        s["pre"] = None
        if case["act"] != "none":                 # what the forward has kept
            p = s["x"].float() @ s["w"].float().T
            s["pre"] = (p if s["bias"] is None else p + s["bias"].float()).bfloat16()
    return s


# ------------------------------------------------------------------ plain forms
def _act(name, p):
    if name == "none":
        return p
    if name == "relu":
        return torch.where(p > 0, p, torch.zeros_like(p))
    if name == "gelu":
        return p * 0.5 * (1 + torch.erf(p * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return p * 0.5 * (1 + torch.tanh((2 / math.pi) ** 0.5 * (p + 0.044715 * p * p * p)))
    return p / (1 + torch.exp(-p))


def _act_slope(name, p):
    if name == "none":
        return torch.ones_like(p)
    if name == "relu":
        return (p > 0).to(p.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(p * 0.5 ** 0.5)) + p * torch.exp(-0.5 * p * p) * (2 * math.pi) ** -0.5
    if name == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (p + 0.044715 * p * p * p))
        return 0.5 * (1 + t) + 0.5 * p * (1 - t * t) * c * (1 + 3 * 0.044715 * p * p)
    s = 1 / (1 + torch.exp(-p))
    return s * (1 + p * (1 - s))


EPS, THETA = 1e-6, 10000.0


def _angles(s):
    """cos and sin [B or 1][1][n][rot / 2]; the angles in 64 bits (far positions)."""
    case = s["case"]
    pos = s["pos"] if s["pos"] is not None else torch.arange(case["n"], device="cuda")[None]
    i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
    a = pos[:, None, :, None].double() * THETA ** (-2 * i / case["rot"])
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(case, x, cos, sin):
    """The first rot features of x turned pair by pair; the rest as they are."""
    r = case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _qk_plain(s):
    cos, sin = _angles(s)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        f = x.float()
        f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w.float()
        out.append(_rotate(s["case"], f, cos, sin).to(x.dtype))
    return out


def _qk_plain_backward(s):
    cos, sin = _angles(s)
    dxs, dws = [], []
    for x, w, dy in ((s["q"], s["wq"], s["dq"]), (s["k"], s["wk"], s["dk"])):
        f = x.float()
        r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
        g = _rotate(s["case"], dy.float(), cos, -sin)
        xhat, dn = f * r, g * w.float()
        dxs.append((r * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))).to(x.dtype))
        dws.append((g * xhat).sum((0, 1, 2)).to(w.dtype))
    return dxs + dws


def _linear_plain(s):
    case = s["case"]
    p = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        p = p + s["bias"].float()
    y = _act(case["act"], p)
    if s["res"] is not None:
        y = y + s["res"].float()
    return [y.bfloat16(), p.bfloat16()] if case["save"] else [y.bfloat16()]


def _linear_plain_backward(s):
    case = s["case"]
    d = s["dy"].float()
    if case["act"] != "none":
        d = d * _act_slope(case["act"], s["pre"].float())
    out = [(d @ s["w"].float()).bfloat16(), (d.T @ s["x"].float()).bfloat16()]
    if case["bias"]:
        out.append(d.sum(0).bfloat16())
    return out


def _gated_plain(s):
    case = s["case"]
    F = case["F"]
    p = s["x"].float() @ s["w"].float().T
    h = (_act(case["act"], p[:, :F]) * p[:, F:]).bfloat16()
    return [h, p.bfloat16()] if case["save"] else [h]


def _gated_plain_backward(s):
    case = s["case"]
    F = case["F"]
    p, d = s["pre"].float(), s["dy"].float()
    gate, up = p[:, :F], p[:, F:]
    dp = torch.cat((d * up * _act_slope(case["act"], gate), d * _act(case["act"], gate)), -1)
    return [(dp @ s["w"].float()).bfloat16(), (dp.T @ s["x"].float()).bfloat16()]


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    from sparse_long_sequence_gb300 import binding as dl
    case = s["case"]
    if case["op"] == "qk":
        how = dict(positions=s["pos"], eps=EPS, theta=THETA, rotary_dim=case["rot"], interleaved=case["interleaved"])
        if case["backward"]:
            return list(dl.diffuser_qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], **how))
        return list(dl.diffuser_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], **how))
    act = getattr(dl, "DIFFUSER_ACT_" + case["act"].upper())
    if case["op"] == "linear":
        if case["backward"]:
            out = dl.diffuser_linear_backward(s["x"], s["w"], s["dy"], pre=s["pre"], activation=act,
                                              with_bias=case["bias"])
            return list(out) if case["bias"] else list(out[:2])
        out = dl.diffuser_linear(s["x"], s["w"], bias=s["bias"], residual=s["res"], activation=act,
                                 save_pre=case["save"])
    else:
        if case["backward"]:
            return list(dl.diffuser_gated_linear_backward(s["x"], s["w"], s["dy"], s["pre"], activation=act))
        out = dl.diffuser_gated_linear(s["x"], s["w"], activation=act, save_pre=case["save"])
    return list(out) if case["save"] else [out]


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    plain = {("qk", False): _qk_plain, ("qk", True): _qk_plain_backward,
             ("linear", False): _linear_plain, ("linear", True): _linear_plain_backward,
             ("gated", False): _gated_plain, ("gated", True): _gated_plain_backward}
    return plain[case["op"], case["backward"]](state)


# ------------------------------------------------------------------ in 64 bits
def _turn64(x, pos, rot, interleaved):
    """Pairs as complex numbers, each times exp(i angle)."""
    ang = pos.double()[:, None, :, None] / THETA ** (torch.arange(0, rot, 2, device=x.device).double() / rot)
    w = torch.polar(torch.ones_like(ang), ang)
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * w
        head = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * w
        head = torch.cat((z.real, z.imag), -1)
    return torch.cat((head, rest), -1)


def _act64(name, p):
    if name == "relu":
        return torch.relu(p)                   # slope 0 at 0
    if name == "gelu":
        return p * torch.special.ndtr(p)
    if name == "gelu_tanh":                    # (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
        return p * torch.sigmoid(math.sqrt(8 / math.pi) * (p + 0.044715 * p ** 3))
    return p * torch.sigmoid(p) if name == "silu" else p


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"] == "qk":
        pos = s["pos"] if s["pos"] is not None else torch.arange(case["n"], device="cuda").expand(case["B"], -1)
        outs, grads, wgrads = [], [], []
        for x, w, dy in (("q", "wq", "dq"), ("k", "wk", "dk")):
            a, b = wide[x].requires_grad_(case["backward"]), wide[w].requires_grad_(case["backward"])
            y = _turn64(a / (a.square().sum(-1, keepdim=True) / HEAD + EPS).sqrt() * b, pos, case["rot"],
                        case["interleaved"])
            outs.append(y.detach())
            if case["backward"]:
                ga, gb = torch.autograd.grad(y, (a, b), wide[dy])
                grads.append(ga)
                wgrads.append(gb)
        return grads + wgrads if case["backward"] else outs
    F, name = case["F"], case["act"]
    if not case["backward"]:
        p = torch.einsum("td,fd->tf", wide["x"], wide["w"])
        if case["op"] == "linear":
            p = p if wide["bias"] is None else p + wide["bias"]
            y = _act64(name, p)
            y = y if wide["res"] is None else y + wide["res"]
        else:
            y = _act64(name, p[:, :F]) * p[:, F:]
        return [y, p] if case["save"] else [y]
    # the slope at the kept pre-activations, then the product's own gradients
    dp = wide["dy"]
    if wide["pre"] is not None:
        p = wide["pre"].requires_grad_(True)
        y = _act64(name, p) if case["op"] == "linear" else _act64(name, p[:, :F]) * p[:, F:]
        dp, = torch.autograd.grad(y, p, wide["dy"])
    x, w = wide["x"].requires_grad_(True), wide["w"].requires_grad_(True)
    dx, dw = torch.autograd.grad(torch.einsum("td,fd->tf", x, w), (x, w), dp)
    return [dx, dw, dp.sum(0)] if case.get("bias") else [dx, dw]
