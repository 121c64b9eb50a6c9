"""The operators around the module (norms with rotation, dense product, gated product),
forward and backward, against their formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-8 is half a bf16 step relative to the value,
e = 2^-24 half an fp32 step):
  * a dot product of K bf16 products in fp32, in any order, with truncating adders:
    at most 2 K e of the sum of the magnitudes;
  * activations: slopes at most 1.13 in magnitude, values and slopes computed within
    2^-18 (|p| + 1): 2^-20 + 2^-24 |p| of the exponential and reciprocal, relative to a factor
    that falls as exp(-|p|) (the second part stays under 2^-25), times |p| in the slope;
  * an element of a product whose left operand was rounded to bf16 (the backward with an
    activation): additionally u times the sum of the magnitudes.  That is the worst case;
    the roundings are independent, so the 2-norm of the error stays under 1.5 u of the
    2-norm of the result (one rounding of the result and one of the operand, each at
    most u / sqrt 3 in the root mean square: 0.82 u together);
  * norms: |x| r w and the rotation in fp32: 16 roundings of values at most the pair's
    norm: 16 e, plus angles within 2^-24 pi; twice that for the backward;
  * a sum of N fp32 values in blocks: N e of the sum of magnitudes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


@pytest.fixture(scope="module")
def dl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_long_sequence_gb300 import binding
    return binding


def act_code(dl, name):
    return getattr(dl, "DIFFUSER_ACT_" + name.upper())


def draw(seed, *shape, scale=1.0, mean=0.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale + mean).to(dtype).cuda()


def act64(name, p):
    if name == "relu":
        return torch.relu(p)                                   # slope 0 at 0, as the library's
    if name == "gelu":
        return p * 0.5 * torch.special.erfc(-p * 0.5 ** 0.5)   # keeps the lower tail's digits
    if name == "gelu_tanh":
        return p * torch.sigmoid((8 / np.pi) ** 0.5 * (p + 0.044715 * p ** 3))
    return p * torch.sigmoid(p) if name == "silu" else p


def slope64(name, p):
    p = p.clone().requires_grad_(True)
    return torch.autograd.grad(act64(name, p).sum(), p)[0] if name != "none" else torch.ones_like(p)


def within(got, ref, tol, what):
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), what
    over = (got.double() - ref).abs() - tol
    assert over.max().item() <= 0, f"{what}: worst excess {over.max().item():.3e} at {over.argmax().item()}"


def near(got, ref, what, limit=1.5 * U):
    norm = ref.norm().item()
    assert (got.double() - ref).norm().item() <= limit * norm + 1e-30, what


# ------------------------------------------------------------------ dense product
SHAPES = [(1, 8, 8), (1, 768, 768), (3, 72, 200), (16, 512, 1368), (17, 1024, 136), (64, 64, 64), (65, 1000, 72),
          (127, 264, 520), (300, 768, 776), (1021, 200, 328), (2100, 136, 1048), (5000, 520, 264),
          (20000, 264, 520), (300, 2056, 4104)]      # several tiles a CTA pair: rows, weight gradients
IDS = ["T%dD%dF%d" % s for s in SHAPES]


def linear_inputs(T, D, F, seed=0, rows=None):
    return draw(seed, T, D), draw(seed + 1, rows or F, D, scale=D ** -0.5), draw(seed + 2, F, scale=0.3)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear(dl, shape, act):
    T, D, F = shape
    X, W, b = linear_inputs(T, D, F, seed=T)
    R = draw(T + 5, T, F)
    x, w = X.double(), W.double()
    p0 = x @ w.T
    mag = x.abs() @ w.abs().T
    for bias, res, save in ((None, None, False), (b, None, True), (None, R, True), (b, R, False)):
        out = dl.diffuser_linear(X, W, bias=bias, residual=res, activation=act_code(dl, act), save_pre=save)
        Y, pre = out if save else (out, None)
        p = p0 if bias is None else p0 + bias.double()
        m = mag if bias is None else mag + bias.double().abs()
        dp = 2 * (D + 2) * E * m
        y = act64(act, p)
        ref = y if res is None else y + res.double()
        slack = 1.13 * dp + (2 ** -18 * (p.abs() + 1) if act != "none" else 0) * (p.abs() > 0)
        within(Y, ref, U * ref.abs() + (1 + U) * slack + 2 * E * (y.abs() + ref.abs()), "Y")
        near(Y, ref, "Y")
        if save:
            within(pre, p, U * p.abs() + (1 + U) * dp, "pre")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear_backward(dl, shape, act):
    T, D, F = shape
    X, W, b = linear_inputs(T, D, F, seed=T)
    dY = draw(T + 7, T, F)
    pre = (X.double() @ W.double().T + b.double()).bfloat16()
    dX, dW, db = dl.diffuser_linear_backward(X, W, dY, pre=None if act == "none" else pre, activation=act_code(dl, act))
    check_linear_backward(X, W, dY, pre, act, dX, dW, db)


def check_linear_backward(X, W, dY, pre, act, dX, dW, db):
    T, D = X.shape
    F = W.shape[0]
    dP = dY.double() * slope64(act, pre.double())
    err = torch.zeros_like(dP)                               # of dP, before its rounding
    if act != "none":
        err = dY.double().abs() * 2 ** -18 * (pre.double().abs() + 1)
    rounded = err + (U * (dP.abs() + err) if act != "none" else 0)
    for got, left, right, k, what in ((dX, dP, W.double(), F, "dX"), (dW, dP.T, X.double(), T, "dW")):
        ref = left @ right
        lerr = rounded if what == "dX" else rounded.T
        slack = lerr @ right.abs() + 2 * (k + 1) * E * ((left.abs() + lerr) @ right.abs())
        within(got, ref, U * ref.abs() + (1 + U) * slack, what)
        near(got, ref, what)
    if db is not None:
        ref = dP.sum(0)
        slack = err.sum(0) + T * E * (dP.abs() + err).sum(0)
        within(db, ref, U * ref.abs() + (1 + U) * slack, "dbias")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", [(1, 8, 8), (1, 72, 4104), (2, 1032, 16), (3, 264, 1000), (4, 64, 520), (4, 2048, 136)], ids=str)
def test_backward_of_few_tokens(dl, shape, act):
    # up to 4 tokens take a kernel of their own, with dP in fp32: one rounding an element
    T, D, F = shape
    X, W, b = linear_inputs(T, D, F, seed=F)
    W2, dY, code = draw(3, 2 * F, D, scale=D ** -0.5), draw(F + 7, T, F), act_code(dl, act)
    pre = (X.double() @ W.double().T + b.double()).bfloat16()
    full = dl.diffuser_linear_backward(X, W, dY, pre=None if act == "none" else pre, activation=code)
    check_linear_backward(X, W, dY, pre, act, *full)
    dP = dY.double() * slope64(act, pre.double())
    for got, ref in zip(full, (dP @ W.double(), dP.T @ X.double(), dP.sum(0))):
        near(got, ref, "few", limit=U)
    for keep in range(8):
        part = dl.diffuser_linear_backward(X, W, dY, pre=pre, activation=code, with_dX=bool(keep & 1),
                                           with_dW=bool(keep & 2), with_bias=bool(keep & 4))
        for bit, (a, f) in enumerate(zip(part, full)):
            assert (a is None) if not keep >> bit & 1 else torch.equal(a, f)
    p2 = (X.double() @ W2.double().T).bfloat16()
    dX, dW = dl.diffuser_gated_linear_backward(X, W2, dY, p2, activation=code)
    g, u = p2.double()[:, :F], p2.double()[:, F:]
    dP = torch.cat((dY.double() * u * slope64(act, g), dY.double() * act64(act, g)), -1)
    near(dX, dP @ W2.double(), "gated dX", limit=U)
    near(dW, dP.T @ X.double(), "gated dW", limit=U)
    again = dl.diffuser_gated_linear_backward(X, W2, dY, p2, activation=code)
    assert torch.equal(dX, again[0]) and torch.equal(dW, again[1])


def test_linear_backward_by_differences(dl):
    # d/dh <dY, Y(X + h V, W + h M, b + h c)> from the forward formula in 64 bits
    T, D, F, act = 19, 40, 48, "gelu"
    X, W, b = linear_inputs(T, D, F, seed=3)
    dY = draw(9, T, F)
    pre = (X.double() @ W.double().T + b.double()).bfloat16()
    dX, dW, db = dl.diffuser_linear_backward(X, W, dY, pre=pre, activation=act_code(dl, act))
    V, M, c = draw(11, T, D).double(), draw(12, F, D).double(), draw(13, F).double()

    def loss(h):
        # the slope is taken at the kept pre-activations
        p = pre.double() + h * (V @ W.double().T + X.double() @ M.T + c)
        return (act64(act, p) * dY.double()).sum()
    h = 1e-5
    want = (loss(h) - loss(-h)) / (2 * h)
    got = (dX.double() * V).sum() + (dW.double() * M).sum() + (db.double() * c).sum()
    # each gradient element off by about u (norm check above): the inner products by u |grad| |direction|
    scale = dX.double().norm() * V.norm() + dW.double().norm() * M.norm() + db.double().norm() * c.norm()
    assert abs(want - got) <= 1.5 * U * scale


def test_linear_parts_and_buffers(dl):
    # any subset of the gradients, given buffers, a leading shape, a residual in place
    X, W, b = linear_inputs(6 * 7, 64, 72, seed=21)
    X3 = X.view(6, 7, 64)
    dY = draw(4, 6, 7, 72)
    pre = dl.diffuser_linear(X3, W, bias=b, save_pre=True)[1]
    code = dl.DIFFUSER_ACT_SILU
    full = dl.diffuser_linear_backward(X3, W, dY, pre=pre, activation=code)
    assert full[0].shape == X3.shape
    for keep in range(8):
        part = dl.diffuser_linear_backward(X3, W, dY, pre=pre, activation=code, with_dX=bool(keep & 1),
                                           with_dW=bool(keep & 2), with_bias=bool(keep & 4))
        for bit, (a, f) in enumerate(zip(part, full)):
            assert (a is None) if not keep >> bit & 1 else torch.equal(a, f)
    R = draw(8, 6, 7, 72)
    want = dl.diffuser_linear(X3, W, bias=b, residual=R, activation=code)
    guard = torch.full((6 * 7 + 2, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = guard[1:-1].view(6, 7, 72)
    Y.copy_(R)
    got = dl.diffuser_linear(X3, W, bias=b, residual=Y, activation=code, Y=Y)
    assert got.data_ptr() == Y.data_ptr() and torch.equal(got, want)
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()          # the rows around it are as they were


# ------------------------------------------------------------------ gated product
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gated_linear(dl, shape, act):
    T, D, F = shape
    X, W, _ = linear_inputs(T, D, F, seed=T + 1, rows=2 * F)
    H, pre = dl.diffuser_gated_linear(X, W, activation=act_code(dl, act), save_pre=True)
    alone = dl.diffuser_gated_linear(X, W, activation=act_code(dl, act))
    assert torch.equal(H, alone)
    p, m = X.double() @ W.double().T, X.double().abs() @ W.double().abs().T
    dp = 2 * (D + 1) * E * m
    g, u, dg, du = p[:, :F], p[:, F:], dp[:, :F], dp[:, F:]
    a = act64(act, g)
    da = 1.13 * dg + (2 ** -18 * (g.abs() + 1) if act != "none" else 0) * (g.abs() > 0)
    ref = a * u
    within(H, ref, U * ref.abs() + (1 + U) * (da * u.abs() + a.abs() * du + da * du + 2 * E * ref.abs()), "H")
    near(H, ref, "H")
    within(pre, p, U * p.abs() + (1 + U) * dp, "pre")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gated_linear_backward(dl, shape, act):
    T, D, F = shape
    X, W, _ = linear_inputs(T, D, F, seed=T + 1, rows=2 * F)
    dH = draw(T + 9, T, F)
    pre = (X.double() @ W.double().T).bfloat16()
    dX, dW = dl.diffuser_gated_linear_backward(X, W, dH, pre, activation=act_code(dl, act))
    p, d = pre.double(), dH.double()
    g, u = p[:, :F], p[:, F:]
    dP = torch.cat((d * u * slope64(act, g), d * act64(act, g)), -1)
    off = 2 ** -18 * (g.abs() + 1) if act != "none" else torch.zeros_like(g)
    err = torch.cat((d.abs() * u.abs() * off, d.abs() * off), -1) + 4 * E * dP.abs()
    rounded = err + U * (dP.abs() + err)
    for got, left, right, k, what in ((dX, dP, W.double(), 2 * F, "dX"), (dW, dP.T, X.double(), T, "dW")):
        ref = left @ right
        lerr = rounded if what == "dX" else rounded.T
        slack = lerr @ right.abs() + 2 * (k + 1) * E * ((left.abs() + lerr) @ right.abs())
        within(got, ref, U * ref.abs() + (1 + U) * slack, what)
        near(got, ref, what)


def test_activation_limits(dl):
    # infinities, NaN, the lowest value and far tails stay in their own row; limits are exact
    lowest = torch.finfo(torch.bfloat16).min
    vals = torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan"), lowest, -lowest, -100.0, 100.0, 1e-30, -20.0,
                         20.0, -8.0, 8.0, -3.0, 3.0], dtype=torch.bfloat16, device="cuda")
    n = vals.numel()
    X = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = vals
    W = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    W[:, 0] = 1
    for act in ACTS:
        Y = dl.diffuser_linear(X, W, activation=act_code(dl, act))[:, 0].float().cpu()
        v = vals.float().cpu()
        want = {"none": v, "relu": torch.relu(v)}.get(act)
        if want is None:
            want = act64(act, v.double())
            want = torch.where(v == float("-inf"), torch.zeros_like(want), want).float()
        assert torch.equal(torch.isnan(Y), torch.isnan(want)), act
        fine = ~torch.isnan(want)
        inf = torch.isinf(want) | (want.abs() >= 3e38)
        assert torch.equal(Y[fine & inf].sign(), want[fine & inf].sign())
        rest = fine & ~inf
        tiny = 2.0 ** -120                                     # the exponential flushes below that
        assert ((Y - want).abs()[rest] <= 1.01 * U * want.abs()[rest] + tiny).all(), (act, Y, want)
        # the slopes at the same places, through a unit gradient
        pre = vals[:, None].expand(n, 8).contiguous()
        one = torch.ones(n, 8, dtype=torch.bfloat16, device="cuda")
        eye = torch.eye(8, dtype=torch.bfloat16, device="cuda")
        dX = dl.diffuser_linear_backward(X, eye, one, pre=pre, activation=act_code(dl, act), with_dW=False,
                                         with_bias=False)[0][:, 0].float().cpu()
        keep = ~torch.isnan(v)
        s = slope64(act, v.double()[keep]) if act != "none" else torch.ones_like(v.double()[keep])
        far = torch.isinf(v[keep]) | (v[keep].abs() > 1e30)
        s[far] = 1.0 if act == "none" else (v[keep][far] > 0).double()
        assert ((dX[keep].double() - s).abs() <= 1.01 * U * s.abs() + 2 ** -18 * (1 + v[keep].double().abs().clamp(max=32)) + tiny).all(), act


# ------------------------------------------------------------------ norms and rotation
def turn64(x, pos, rot, interleaved, theta, sign=1):
    ang = sign * pos.double()[:, None, :, None] * theta ** (-torch.arange(0, rot, 2, device=x.device).double() / rot)
    z = torch.polar(torch.ones_like(ang), ang)
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        t = torch.view_as_real(torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * z)
        head = t.reshape(head.shape)
    else:
        t = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * z
        head = torch.cat((t.real, t.imag), -1)
    return torch.cat((head, rest), -1)


QK = [  # B, Hq, Hk, n, rot, interleaved, weights, far
    (1, 1, 1, 1, 64, False, True, False),
    (2, 3, 1, 5, 64, True, True, True),
    (1, 12, 12, 257, 64, False, True, False),
    (3, 4, 2, 77, 32, False, True, True),
    (2, 5, 7, 33, 48, False, False, True),
    (2, 2, 2, 130, 16, True, True, True),
    (16, 16, 16, 1, 64, False, True, True),
    (1, 2, 3, 1025, 0, False, True, False),
    (4, 1, 8, 1000, 48, True, False, True),
    (1, 16, 16, 4096, 64, False, True, False),
]


def qk_case(case, dtype):
    B, Hq, Hk, n, rot, inter, weights, far = case
    q, k = draw(n, B, Hq, n, 64, dtype=dtype), draw(n + 1, B, Hk, n, 64, dtype=dtype)
    wq = draw(5, 64, scale=0.3, mean=1.0, dtype=dtype) if weights else None
    wk = draw(6, 64, scale=0.3, mean=1.0, dtype=dtype) if weights else None
    pos = None
    if far:
        g = torch.Generator().manual_seed(n)
        pos = torch.randint(-(1 << 31), 1 << 31, (B, n), generator=g).cuda()
    return q, k, wq, wk, pos, dict(eps=1e-5, theta=10000.0, rotary_dim=rot, interleaved=inter)


def positions64(pos, B, n, offset):
    base = torch.arange(n, device="cuda").expand(B, n) if pos is None else pos
    return base + offset


def norm64(x, w, eps):
    xh = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return xh if w is None else xh * w


def angle_error(pos):
    # the reference's own angle is a 64-bit product: half a step of up to 2^32 radians
    return np.pi * 2 ** -24 + pos.abs().max().item() * 2 ** -52


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", QK, ids=str)
def test_qk_norm_rope(dl, case, dtype):
    q, k, wq, wk, pos, how = qk_case(case, dtype)
    B, n = q.shape[0], q.shape[2]
    offset = 0 if case[-1] else 4000
    Qo, Ko = dl.diffuser_qk_norm_rope(q, k, wq, wk, positions=pos, position_offset=offset, **how)
    at = positions64(pos, B, n, offset)
    for got, x, w in ((Qo, q, wq), (Ko, k, wk)):
        y = norm64(x.double(), None if w is None else w.double(), how["eps"])
        ref = turn64(y, at, how["rotary_dim"], how["interleaved"], how["theta"]) if how["rotary_dim"] else y
        size = y.abs().amax(-1, keepdim=True) * 2 ** 0.5
        tol = (16 * E + angle_error(at)) * size
        within(got, ref, tol + (U * (ref.abs() + tol) if dtype == torch.bfloat16 else 0), "y")
    # in place
    q2, k2 = q.clone(), k.clone()
    dl.diffuser_qk_norm_rope(q2, k2, wq, wk, positions=pos, position_offset=offset, Qo=q2, Ko=k2, **how)
    assert torch.equal(q2, Qo) and torch.equal(k2, Ko)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", QK, ids=str)
def test_qk_norm_rope_backward(dl, case, dtype):
    q, k, wq, wk, pos, how = qk_case(case, dtype)
    B, n = q.shape[0], q.shape[2]
    dq, dk = draw(n + 2, *q.shape, dtype=dtype), draw(n + 3, *k.shape, dtype=dtype)
    got = dl.diffuser_qk_norm_rope_backward(q, k, dq, dk, wq, wk, positions=pos, **how)
    again = dl.diffuser_qk_norm_rope_backward(q, k, dq, dk, wq, wk, positions=pos, **how)
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)
    at = positions64(pos, B, n, 0)
    for dx, dw, x, w, dy in ((got[0], got[2], q, wq, dq), (got[1], got[3], k, wk, dk)):
        a = x.double().requires_grad_(True)
        b = (torch.ones(64, device="cuda") if w is None else w).double().requires_grad_(True)
        y = norm64(a, b, how["eps"])
        if how["rotary_dim"]:
            y = turn64(y, at, how["rotary_dim"], how["interleaved"], how["theta"])
        ra, rb = torch.autograd.grad(y, (a, b), dy.double())
        r = (x.double().square().mean(-1, keepdim=True) + how["eps"]).rsqrt()
        xh = x.double() * r
        g = dy.double().abs().amax(-1, keepdim=True) * 2 ** 0.5
        size = r * g * b.detach().abs().max() * (1 + xh.abs() * xh.abs().mean(-1, keepdim=True))
        rel = 2 * (16 * E + angle_error(at)) + 64 * E
        tol = rel * size
        within(dx, ra, tol + (U * (ra.abs() + tol) if dtype == torch.bfloat16 else 0), "dx")
        if w is None:
            assert dw is None
        else:
            mag = (g * xh.abs()).sum((0, 1, 2))
            # at most (units of a warp x its heads) + 8 + 76 + 8 additions of fp32 values in a row
            tol = (rel + 512 * E) * mag
            within(dw, rb, tol + (U * (rb.abs() + tol) if dtype == torch.bfloat16 else 0), "dw")


def test_qk_rotation_keeps_relative_positions(dl):
    # q.k after rotation depends on the distance alone: shifting both positions changes nothing
    q, k = draw(1, 1, 2, 50, 64, dtype=torch.float32), draw(2, 1, 2, 50, 64, dtype=torch.float32)
    def scores(offset):
        a, b = dl.diffuser_qk_norm_rope(q, k, position_offset=offset)
        return a.double() @ b.double().transpose(-1, -2)
    near0 = scores(0)
    for offset in (1, 4095, 1 << 20, (1 << 31) + 5, -(1 << 40)):
        # 64 products of values whose turn is off by at most 2^-24 pi + 16 e each
        assert (scores(offset) - near0).abs().max().item() <= 2 * 64 * (16 * E + np.pi * 2 ** -24) * 8


def test_qk_rows_of_zeros_and_extremes(dl):
    for dtype in (torch.float32, torch.bfloat16):
        q = draw(3, 1, 2, 9, 64, dtype=dtype)
        clean = dl.diffuser_qk_norm_rope(q, q.clone())[0]
        q2 = q.clone()
        q2[0, 0, 2] = 0
        q2[0, 0, 4] = float("nan")
        q2[0, 0, 6, 3] = float("inf")
        out = dl.diffuser_qk_norm_rope(q2, q2.clone())[0]
        assert (out[0, 0, 2] == 0).all()
        assert torch.isnan(out[0, 0, 4]).all() and torch.isnan(out[0, 0, 6]).any()
        keep = [t for t in range(9) if t not in (2, 4, 6)]
        assert torch.equal(out[0, 0, keep], clean[0, 0, keep]) and torch.equal(out[0, 1], clean[0, 1])
        grads = dl.diffuser_qk_norm_rope_backward(torch.zeros_like(q), torch.zeros_like(q), q, q)
        assert torch.isfinite(grads[0]).all() and torch.isfinite(grads[1]).all()


@pytest.mark.parametrize("shape", [(3, 65536, 8), (70, 65536, 16), (3, 8, 65536), (70, 8, 65536), (270, 24, 32776)], ids=str)
def test_widest(dl, shape):
    T, D, F = shape
    X, W, b = linear_inputs(T, D, F, seed=F)
    W2, dY, code = draw(3, 2 * F, D, scale=D ** -0.5), draw(F + 7, T, F), dl.DIFFUSER_ACT_SILU
    Y, pre = dl.diffuser_linear(X, W, bias=b, activation=code, save_pre=True)
    p = X.double() @ W.double().T + b.double()
    dp = 2 * (D + 2) * E * (X.double().abs() @ W.double().abs().T + b.double().abs())
    within(pre, p, U * p.abs() + (1 + U) * dp, "pre")
    near(Y, act64("silu", p), "Y")
    ws = torch.empty(dl.diffuser_linear_backward_workspace_size(T, D, F, code), dtype=torch.uint8, device="cuda")
    check_linear_backward(X, W, dY, pre, "silu", *dl.diffuser_linear_backward(X, W, dY, pre=pre, activation=code,
                                                                              workspace=ws if ws.numel() else None))
    H, gu = dl.diffuser_gated_linear(X, W2, save_pre=True)
    q = X.double() @ W2.double().T
    near(H, act64("silu", q[:, :F]) * q[:, F:], "H")
    dX, dW = dl.diffuser_gated_linear_backward(X, W2, dY, gu)
    g, u, d = gu.double()[:, :F], gu.double()[:, F:], dY.double()
    dP = torch.cat((d * u * slope64("silu", g), d * act64("silu", g)), -1)
    near(dX, dP @ W2.double(), "gated dX")
    near(dW, dP.T @ X.double(), "gated dW")


def test_qk_of_many_heads(dl):
    q, k = draw(1, 1, 4096, 3, 64), draw(2, 1, 2, 3, 64)
    w = draw(3, 64, mean=1.0)
    Qo, Ko = dl.diffuser_qk_norm_rope(q, k, w, w, position_offset=77)
    for h in (0, 1, 2047, 4095):
        one = q[:, h:h + 1].contiguous()
        assert torch.equal(Qo[:, h:h + 1], dl.diffuser_qk_norm_rope(one, one.clone(), w, w, position_offset=77)[0])
    dQ, _, dw, _ = dl.diffuser_qk_norm_rope_backward(q, k, Qo, Ko, w, w, position_offset=77)
    # dy = y: g is the normed and weighted row, so dw = sum of w xh^2
    xh = norm64(q.double(), None, 1e-6)
    ref = (w.double() * xh.square()).sum((0, 1, 2))
    mag = ref.abs()
    within(dw, ref, U * mag + 2 * U * mag, "dw")          # its own rounding, and that of y


# ------------------------------------------------------------------ where they write
def guarded(rows, width, dtype=torch.bfloat16, fill=7.0):
    """A [rows][width] buffer between rows of `fill`, and a check that those are as they were."""
    whole = torch.full((rows + 4, width), fill, dtype=dtype, device="cuda")
    inner = whole[2:rows + 2]
    return inner, lambda: bool((whole[:2] == fill).all() and (whole[-2:] == fill).all())


@pytest.mark.parametrize("shape", [(1, 64, 72), (3, 200, 88), (19, 136, 88), (130, 72, 200), (2050, 200, 136), (20010, 72, 520),
                                   (700, 2056, 328)], ids=lambda s: "T%dD%dF%d" % s)
def test_nothing_is_written_outside(dl, shape):
    T, D, F = shape
    X, W, b = linear_inputs(T, D, F, seed=T)
    W2 = draw(7, 2 * F, D, scale=D ** -0.5)
    R, dY, code = draw(8, T, F), draw(9, T, F), dl.DIFFUSER_ACT_SILU
    (Y, y_ok), (P, p_ok) = guarded(T, F), guarded(T, F)
    dl.diffuser_linear(X, W, bias=b, residual=R, activation=code, Y=Y, pre=P)
    want = dl.diffuser_linear(X, W, bias=b, residual=R, activation=code, save_pre=True)
    assert y_ok() and p_ok() and torch.equal(Y, want[0]) and torch.equal(P, want[1])
    (dX, dx_ok), (dW, dw_ok), (db, db_ok) = guarded(T, D), guarded(F, D), guarded(1, F)
    dl.diffuser_linear_backward(X, W, dY, pre=P, activation=code, dX=dX, dW=dW, dbias=db[0])
    assert dx_ok() and dw_ok() and db_ok()
    check_linear_backward(X, W, dY, P, "silu", dX, dW, db[0])
    (H, h_ok), (G, g_ok) = guarded(T, F), guarded(T, 2 * F)
    dl.diffuser_gated_linear(X, W2, H=H, pre=G)
    want = dl.diffuser_gated_linear(X, W2, save_pre=True)
    assert h_ok() and g_ok() and torch.equal(H, want[0]) and torch.equal(G, want[1])
    (dX, dx_ok), (dW, dw_ok) = guarded(T, D), guarded(2 * F, D)
    dl.diffuser_gated_linear_backward(X, W2, dY, G, dX=dX, dWgu=dW)
    again = dl.diffuser_gated_linear_backward(X, W2, dY, G)
    assert dx_ok() and dw_ok() and torch.equal(dX, again[0]) and torch.equal(dW, again[1])


def test_qk_writes_only_its_rows(dl):
    for dtype in (torch.float32, torch.bfloat16):
        for n in (1, 5, 33):
            q, k = draw(1, 1, 2, n, 64, dtype=dtype), draw(2, 1, 3, n, 64, dtype=dtype)
            outs = [guarded(r, 64, dtype) for r in (2 * n, 3 * n)]
            dl.diffuser_qk_norm_rope(q, k, Qo=outs[0][0].view(1, 2, n, 64), Ko=outs[1][0].view(1, 3, n, 64))
            assert all(ok() for _, ok in outs)
            w = draw(3, 64, dtype=dtype)
            small = [guarded(1, 64, dtype) for _ in range(2)]
            dl.diffuser_qk_norm_rope_backward(q, k, q, k, w, w, dQ=outs[0][0].view(1, 2, n, 64),
                                              dK=outs[1][0].view(1, 3, n, 64), dq_weight=small[0][0][0],
                                              dk_weight=small[1][0][0])
            assert all(ok() for _, ok in outs + small)


def test_offsets_past_32_bits(dl):
    # results of more than 2^31 elements: their last rows against the same rows alone
    T, D, F = 600_011, 64, 4096
    g = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(T, D, generator=g, device="cuda", dtype=torch.bfloat16)
    W, b = draw(1, F, D, scale=D ** -0.5), draw(2, F)
    tail = X[-300:].contiguous()
    Y, P = dl.diffuser_linear(X, W, bias=b, activation=dl.DIFFUSER_ACT_GELU, save_pre=True)
    y, p = dl.diffuser_linear(tail, W, bias=b, activation=dl.DIFFUSER_ACT_GELU, save_pre=True)
    assert Y.numel() > 2 ** 31 and torch.equal(Y[-300:], y) and torch.equal(P[-300:], p)
    dX = dl.diffuser_linear_backward(X, W, Y, pre=P, activation=dl.DIFFUSER_ACT_GELU, with_dW=False, with_bias=False)[0]
    dx = dl.diffuser_linear_backward(tail, W, y, pre=p, activation=dl.DIFFUSER_ACT_GELU, with_dW=False, with_bias=False)[0]
    near(dX[-300:], dx.double(), "dX")                    # another split of K, another order of the sum
    del Y, P, dX
    B, H, n = 1, 17, 2_000_003
    q = torch.randn(B, H, n, 64, generator=g, device="cuda", dtype=torch.bfloat16)
    k = q.new_zeros(B, 1, n, 64)
    Q, _ = dl.diffuser_qk_norm_rope(q, k)
    assert q.numel() > 2 ** 31
    last = q[:, -1:, -40:].contiguous()
    want = dl.diffuser_qk_norm_rope(last, last.clone(), position_offset=n - 40)[0]
    assert torch.equal(Q[:, -1:, -40:], want)
    dQ = dl.diffuser_qk_norm_rope_backward(q, k, Q, k)[0]
    wd = dl.diffuser_qk_norm_rope_backward(last, last.clone(), want, last.clone(), position_offset=n - 40)[0]
    assert torch.equal(dQ[:, -1:, -40:], wd)


# ------------------------------------------------------------------ how they are called
def test_empty_and_single(dl):
    X, W = draw(0, 0, 64), draw(1, 72, 64)
    assert dl.diffuser_linear(X, W).shape == (0, 72)
    dX, dW, db = dl.diffuser_linear_backward(X, W, draw(0, 0, 72))
    assert dX.shape == (0, 64) and not dW.any() and not db.any()
    W2 = draw(1, 144, 64)
    assert dl.diffuser_gated_linear(X, W2).shape == (0, 72)
    dX, dW = dl.diffuser_gated_linear_backward(X, W2, draw(0, 0, 72), draw(0, 0, 144))
    assert not dW.any()
    q = draw(0, 2, 3, 0, 64)
    w = draw(1, 64)
    assert dl.diffuser_qk_norm_rope(q, q.clone(), w, w)[0].shape == q.shape
    out = dl.diffuser_qk_norm_rope_backward(q, q.clone(), q.clone(), q.clone(), w, w.clone())
    assert not out[2].any() and not out[3].any()
    x = draw(4, 64)                                                    # one row without a leading shape
    assert torch.equal(dl.diffuser_linear(x, W), dl.diffuser_linear(x[None], W)[0])


def test_refusals_of_the_binding(dl):
    X, W, b = linear_inputs(5, 64, 72)
    before = dl.diffuser_launch_count()[0]
    bad = [lambda: dl.diffuser_linear(X.float(), W), lambda: dl.diffuser_linear(X, W.float()),
           lambda: dl.diffuser_linear(X, W.T), lambda: dl.diffuser_linear(X, W[:, :32]),
           lambda: dl.diffuser_linear(X, W, bias=b[:8]), lambda: dl.diffuser_linear(X, W, residual=X),
           lambda: dl.diffuser_linear(X.T.contiguous().T, W), lambda: dl.diffuser_linear(X, W.cpu()),
           lambda: dl.diffuser_linear(X.cpu(), W), lambda: dl.diffuser_linear(X, W, activation=9),
           lambda: dl.diffuser_linear(X[:, :12].contiguous(), W[:, :12].contiguous()),
           lambda: dl.diffuser_linear(X, W, Y=X), lambda: dl.diffuser_linear(X, W[:64], Y=X),
           lambda: dl.diffuser_linear_backward(X, W, draw(1, 5, 72), activation=1),
           lambda: dl.diffuser_linear_backward(X, W, draw(1, 5, 72), workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: dl.diffuser_gated_linear(X, W[:71]),
           lambda: dl.diffuser_gated_linear_backward(X, W, draw(1, 5, 36), draw(1, 5, 36))]
    q = draw(1, 1, 2, 5, 64)
    bad += [lambda: dl.diffuser_qk_norm_rope(q, q.float()), lambda: dl.diffuser_qk_norm_rope(q, q[:, :, :4]),
            lambda: dl.diffuser_qk_norm_rope(q, q, rotary_dim=24), lambda: dl.diffuser_qk_norm_rope(q, q, eps=0.0),
            lambda: dl.diffuser_qk_norm_rope(q, q, theta=0.5),
            lambda: dl.diffuser_qk_norm_rope(q, q, positions=torch.zeros(1, 5, device="cuda", dtype=torch.int32)),
            lambda: dl.diffuser_qk_norm_rope(q, q, positions=torch.zeros(5, device="cuda", dtype=torch.int64)),
            lambda: dl.diffuser_qk_norm_rope(q, q, Qo=q, Ko=q),
            lambda: dl.diffuser_qk_norm_rope(q[..., :32].contiguous(), q[..., :32].contiguous()),
            lambda: dl.diffuser_qk_norm_rope_backward(q, q.clone(), q.clone(), q.clone(), dQ=q)]
    for k, call in enumerate(bad):
        with pytest.raises((dl.DiffuserError, ValueError, TypeError)):
            call()
            pytest.fail(f"call {k} was accepted")
    assert dl.diffuser_launch_count()[0] == before
    assert dl.diffuser_projection_status() == 0


def layer(dl, g, P, X, save=False):
    """A transformer layer around the module, as its user writes it."""
    B, n, D = X.shape
    H = D // 64
    Q, K, V = dl.diffuser_qkv_projection(X, P["qkv"], H)
    Q, K = dl.diffuser_qk_norm_rope(Q, K, P["nq"], P["nk"], Qo=Q, Ko=K)
    Z = dl.diffuser_forward(Q, K, V, g, 3, 0.1)
    heads = Z.transpose(1, 2).reshape(B, n, D)
    A = dl.diffuser_linear(heads, P["o"], bias=P["ob"], residual=X)
    F = dl.diffuser_gated_linear(A, P["gu"])
    return dl.diffuser_linear(F, P["down"], residual=A)


def layer_weights(D, F, seed=1):
    H = D // 64
    return dict(qkv=draw(seed, 3 * H * 64, D, scale=D ** -0.5), nq=draw(seed + 1, 64, scale=0.2, mean=1.0),
                nk=draw(seed + 2, 64, scale=0.2, mean=1.0), o=draw(seed + 3, D, D, scale=D ** -0.5),
                ob=draw(seed + 4, D, scale=0.1), gu=draw(seed + 5, 2 * F, D, scale=D ** -0.5),
                down=draw(seed + 6, D, F, scale=F ** -0.5))


def test_layer_of_them_together(dl):
    B, n, D, F = 2, 300, 128, 344
    H = D // 64
    g = dl.diffuser_build_graph(n, 16, 3, rand_per_row=5, seed=0)
    row_ptr, col = dl.diffuser_graph_copy_csr(g)
    P = layer_weights(D, F)
    X = draw(40, B, n, D)
    Y = layer(dl, g, P, X)
    # the formulas in 64 bits, each tensor between the stages rounded to bf16 once
    w = {k: v.double() for k, v in P.items()}
    r = lambda t: t.bfloat16().double()
    x = X.double()
    q, k, v = (r(x @ w["qkv"].T).view(B, n, 3, H, 64).permute(2, 0, 3, 1, 4))
    pos = torch.arange(n, device="cuda").expand(B, n)
    q, k = (r(turn64(norm64(t, w[m], 1e-6), pos, 64, False, 10000.0)) for t, m in ((q, "nq"), (k, "nk")))
    mask = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        mask[i, torch.from_numpy(col[row_ptr[i]:row_ptr[i + 1]].astype(np.int64))] = True
    s = (q @ k.transpose(-1, -2) / 8).masked_fill(~mask.cuda(), float("-inf"))
    a = torch.softmax(s, -1)
    z = v
    for _ in range(3):
        z = 0.9 * (a @ z) + 0.1 * v
    heads = r(z).transpose(1, 2).reshape(B, n, D)
    A = r(x + heads @ w["o"].T + w["ob"])
    gu = A @ w["gu"].T
    h = r(act64("silu", gu[..., :F]) * gu[..., F:])
    ref = A + h @ w["down"].T
    # the roundings between the stages fall alike but for values next to a border: each
    # stage adds at most its own half step, eight of them
    near(Y, ref, "layer", limit=8 * U)


def test_two_captured_graphs_and_streams(dl):
    # one capture per stream without shared workspaces, replayed on new inputs, at the same
    # time, give what eager calls give
    D, F, T = 128, 264, 70
    X, W, b = linear_inputs(T, D, F, seed=2)
    W2 = draw(8, 2 * F, D, scale=D ** -0.5)
    q, k = draw(3, 2, 2, T, 64), draw(4, 2, 2, T, 64)
    w = draw(5, 64, mean=1.0)
    dY = draw(6, T, F)

    def run(x):
        y, pre = dl.diffuser_linear(x, W, bias=b, activation=dl.DIFFUSER_ACT_GELU, save_pre=True)
        grads = dl.diffuser_linear_backward(x, W, dY, pre=pre, activation=dl.DIFFUSER_ACT_GELU)
        h, gu = dl.diffuser_gated_linear(x, W2, save_pre=True)
        ggrads = dl.diffuser_gated_linear_backward(x, W2, dY, gu)
        qk = dl.diffuser_qk_norm_rope(q, k, w, w)
        qg = dl.diffuser_qk_norm_rope_backward(q, k, q, k, w, w)
        return [y, pre, *grads, h, gu, *ggrads, *qk, *qg]
    xs = [X.clone(), X.flip(0).contiguous()]
    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x, s in zip(xs, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs.append(run(x))
        graphs.append(gr)
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        for a, c in zip(got, ref):
            assert torch.equal(a, c)
    # an explicit stream, the outputs allocated on it
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = dl.diffuser_linear(xs[0], W, bias=b, activation=dl.DIFFUSER_ACT_GELU, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0][0])


def test_calls_at_once_on_two_streams(dl):
    # large products that fill the GPU, on two streams without waits between them
    X, W, b = linear_inputs(5000, 264, 776, seed=31)
    X2, W2, _ = linear_inputs(4100, 520, 392, seed=37, rows=784)
    dY, dH = draw(1, 5000, 776), draw(2, 4100, 392)

    def one():
        y, p = dl.diffuser_linear(X, W, bias=b, activation=dl.DIFFUSER_ACT_RELU, save_pre=True)
        return [y, p, *dl.diffuser_linear_backward(X, W, dY, pre=p, activation=dl.DIFFUSER_ACT_RELU)]

    def two():
        h, p = dl.diffuser_gated_linear(X2, W2, save_pre=True)
        return [h, p, *dl.diffuser_gated_linear_backward(X2, W2, dH, p)]
    want = one(), two()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(10):
        for k, (s, f) in enumerate(zip(streams, (one, two))):
            with torch.cuda.stream(s):
                got[k].append(f())
    torch.cuda.synchronize()
    for outs, ref in zip(got, want):
        for out in outs:
            assert all(torch.equal(a, c) for a, c in zip(out, ref))


@pytest.mark.parametrize("rows", [5, 300, 3000])
def test_first_call_inside_a_capture(dl, rows):
    # a new process whose first calls of all are captured: the status block and the kernels'
    # attributes are made outside the capture
    import os
    import subprocess
    import sys
    code = f"""
import torch
from sparse_long_sequence_gb300 import binding as dl
r = lambda *s: torch.randn(*s, device='cuda').bfloat16()
x, w, w2, dy, q = r({rows}, 64), r(264, 64), r(528, 64), r({rows}, 264), r(1, 2, {rows}, 64)
torch.cuda.synchronize()
def run():
    y, p = dl.diffuser_linear(x, w, activation=dl.DIFFUSER_ACT_GELU, save_pre=True)
    h, gu = dl.diffuser_gated_linear(x, w2, save_pre=True)
    return [y, p, h, gu, *dl.diffuser_linear_backward(x, w, dy, pre=p, activation=dl.DIFFUSER_ACT_GELU),
            *dl.diffuser_gated_linear_backward(x, w2, dy, gu), *dl.diffuser_qk_norm_rope(q, q.clone()),
            *dl.diffuser_qk_norm_rope_backward(q, q.clone(), q.clone(), q.clone())[:2]]
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


def test_status_word_is_clear(dl):
    X, W, _ = linear_inputs(5, 64, 72)
    assert dl.diffuser_projection_status(reset=True) == 0
    dl.diffuser_linear(X, W)
    torch.cuda.synchronize()
    assert dl.diffuser_projection_status() == 0
