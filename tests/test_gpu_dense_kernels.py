"""Every kernel that the dense products' rule can pick, at sizes where it picks it whatever number
of clusters the device holds (tests/dense_sizes.py), against the formulas in 64 bits, with the
bounds that tests/test_gpu_layer_ops.py derives; and the activations' values and slopes at their
limits on each of them.

Tails (relative): a slope or value far below 0 is a product of the exponential, of fp32 sums
without cancellation and of the value's rounding to bf16, U.  The exponential's argument is up to
127 in units of log 2, rounded to 2^-24 of itself (2^-17 of the result), its own error and the
reciprocal's are 2^-21 each, and gelu's and gelu_tanh's arguments are products of up to four
factors (another 2^-17 each): under 2^-15.  Below 2^-126 the exponential or the reciprocal is 0,
which |p| and the inner slope enlarge to at most 2^-116.
"""
import pytest

from tests import dense_sizes as sizes
from tests.test_gpu_layer_ops import (ACTS, E, U, act64, act_code, check_linear_backward, dl, draw, linear_inputs, near,
                                      slope64, within)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def cases(table):
    out = [(kernel, shape) for kernel, shapes in table.items() for shape in shapes]
    return pytest.mark.parametrize("kernel,shape", out, ids=["-".join(map(str, k)) + "-T%dD%dF%d" % s for k, s in out])


@cases(sizes.FORWARD)
def test_forward(dl, kernel, shape):
    T, D, F = shape
    X, W, b = linear_inputs(T, D, F, seed=T)
    R = draw(T + 5, T, F)
    x, w = X.double(), W.double()
    p0, mag = x @ w.T, x.abs() @ w.abs().T
    for k, (bias, res, save) in enumerate(((b, R, True), (b, R, False), (None, R, True), (None, R, False), (b, None, True),
                                           (None, None, False), (None, None, True))):
        act = ACTS[(k + F // 8) % len(ACTS)]
        out = dl.diffuser_linear(X, W, bias=bias, residual=res, activation=act_code(dl, act), save_pre=save)
        Y, pre = out if save else (out, None)
        p = p0 if bias is None else p0 + bias.double()
        dp = 2 * (D + 2) * E * (mag if bias is None else mag + bias.double().abs())
        y = act64(act, p)
        ref = y if res is None else y + res.double()
        slack = 1.13 * dp + (2 ** -18 * (p.abs() + 1) if act != "none" else 0) * (p.abs() > 0)
        within(Y, ref, U * ref.abs() + (1 + U) * slack + 2 * E * (y.abs() + ref.abs()), "Y")
        near(Y, ref, "Y")
        if save:
            within(pre, p, U * p.abs() + (1 + U) * dp, "pre")
        if res is not None:                                      # in place, between rows of another value
            whole = torch.full((T + 4, F), 7.0, dtype=torch.bfloat16, device="cuda")
            inner = whole[2:T + 2]
            inner.copy_(R)
            again = dl.diffuser_linear(X, W, bias=bias, residual=inner, activation=act_code(dl, act), Y=inner, save_pre=save)
            assert torch.equal(inner, Y) and (not save or torch.equal(again[1], pre))
            assert (whole[:2] == 7).all() and (whole[-2:] == 7).all()


@cases(sizes.GATED)
def test_gated(dl, kernel, shape):
    T, D, F = shape
    X, W, _ = linear_inputs(T, D, F, seed=T + 1, rows=2 * F)
    p, m = X.double() @ W.double().T, X.double().abs() @ W.double().abs().T
    dp = 2 * (D + 1) * E * m
    g, u, dg, du = p[:, :F], p[:, F:], dp[:, :F], dp[:, F:]
    for act in ACTS[1:]:
        H, pre = dl.diffuser_gated_linear(X, W, activation=act_code(dl, act), save_pre=True)
        assert torch.equal(H, dl.diffuser_gated_linear(X, W, activation=act_code(dl, act)))
        a = act64(act, g)
        da = 1.13 * dg + 2 ** -18 * (g.abs() + 1) * (g.abs() > 0)
        ref = a * u
        within(H, ref, U * ref.abs() + (1 + U) * (da * u.abs() + a.abs() * du + da * du + 2 * E * ref.abs()), "H")
        near(H, ref, "H")
        within(pre, p, U * p.abs() + (1 + U) * dp, "pre")


def backward(dl, shape, **parts):
    T, D, F = shape
    X, W, b = linear_inputs(T, D, F, seed=T)
    dY = draw(T + 7, T, F)
    pre = (X.double() @ W.double().T + b.double()).bfloat16()
    for act in ("none", ACTS[1 + F // 8 % 4]):
        out = dl.diffuser_linear_backward(X, W, dY, pre=None if act == "none" else pre, activation=act_code(dl, act), **parts)
        yield X, W, dY, pre, act, out


@cases(sizes.INPUT_GRADIENT)
def test_input_gradient(dl, kernel, shape):
    for X, W, dY, pre, act, (dX, dW, db) in backward(dl, shape, with_dW=False):
        assert dW is None
        dP = dY.double() * slope64(act, pre.double())
        err = dY.double().abs() * 2 ** -18 * (pre.double().abs() + 1) if act != "none" else torch.zeros_like(dP)
        off = err + (U * (dP.abs() + err) if act != "none" else 0)
        w = W.double()
        ref, slack = dP @ w, off @ w.abs() + 2 * (shape[2] + 1) * E * ((dP.abs() + off) @ w.abs())
        within(dX, ref, U * ref.abs() + (1 + U) * slack, "dX")
        near(dX, ref, "dX")
        sums = dP.sum(0)
        within(db, sums, U * sums.abs() + (1 + U) * (err.sum(0) + shape[0] * E * (dP.abs() + err).sum(0)), "dbias")


@cases(sizes.WEIGHT_GRADIENT)
def test_weight_gradient(dl, kernel, shape):
    for X, W, dY, pre, act, (dX, dW, db) in backward(dl, shape, with_dX=False, with_bias=False):
        assert dX is None and db is None
        dP = dY.double() * slope64(act, pre.double())
        err = dY.double().abs() * 2 ** -18 * (pre.double().abs() + 1) if act != "none" else torch.zeros_like(dP)
        off = err + (U * (dP.abs() + err) if act != "none" else 0)
        x = X.double()
        ref, slack = dP.T @ x, off.T @ x.abs() + 2 * (shape[0] + 1) * E * ((dP.abs() + off).T @ x.abs())
        within(dW, ref, U * ref.abs() + (1 + U) * slack, "dW")
        near(dW, ref, "dW")


@cases(sizes.BOTH_GRADIENTS)
def test_both_gradients(dl, kernel, shape):
    for X, W, dY, pre, act, grads in backward(dl, shape):
        check_linear_backward(X, W, dY, pre, act, *grads)
    T, D, F = shape
    W2, dH = draw(3, F // 16 * 16, D, scale=D ** -0.5), draw(4, T, F // 16 * 8)
    X = draw(T, T, D)
    pre = (X.double() @ W2.double().T).bfloat16()
    dX, dW = dl.diffuser_gated_linear_backward(X, W2, dH, pre, activation=dl.DIFFUSER_ACT_GELU)
    g, u, d = *pre.double().chunk(2, -1), dH.double()
    dP = torch.cat((d * u * slope64("gelu", g), d * act64("gelu", g)), -1)
    near(dX, dP @ W2.double(), "gated dX")
    near(dW, dP.T @ X.double(), "gated dW")


# ------------------------------------------------------------------ limits and tails
LOWEST = torch.finfo(torch.bfloat16).min
BEYOND = [0.0, -0.0, float("inf"), float("-inf"), float("nan"), LOWEST, -LOWEST, -100.0, 100.0, 1e-30]
TAILS = [-0.25, -1.0, -2.0, -3.0, -4.0, -5.0, -6.0, -7.0, -8.0, -9.0, -10.0, -12.0, -13.0, -20.0, -40.0, -60.0, -80.0]
TAILS += [-v for v in TAILS]
REL, TINY = 1.01 * U + 2.0 ** -15, 2.0 ** -116
ONE_OF_EACH = pytest.mark.parametrize("kernel", [k for k in sizes.FORWARD], ids=lambda k: "-".join(map(str, k)))


def spread(values, T):
    """Every value over the tokens, and the token's value."""
    v = torch.tensor(values, dtype=torch.bfloat16)
    return v[torch.arange(T) % len(v)].cuda()


def check_values(got, act, v):
    """got [T][F]: act(v) in every column."""
    assert ((got == got[:, :1]) | (got.isnan() & got[:, :1].isnan())).all()
    got, v = got[:, 0].double(), v.double()
    want = act64(act, v) if act != "none" else v
    want = torch.where(v == float("-inf"), want if act == "none" else torch.zeros_like(v), want)
    assert torch.equal(got.isnan(), want.isnan()), act
    huge = want.abs() >= 3e38
    assert torch.equal(got[huge].sign(), want[huge].sign()) and (got[huge].abs() >= 3e38).all()
    rest = ~huge & ~want.isnan()
    assert ((got - want).abs()[rest] <= REL * want.abs()[rest] + TINY).all(), (act, v[rest], got[rest], want[rest])


@ONE_OF_EACH
def test_values_at_limits(dl, kernel):
    T, D, F = max(sizes.FORWARD[kernel], key=lambda s: s[0])
    v = spread(BEYOND + TAILS, T)
    X, W = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(F, D, dtype=torch.bfloat16, device="cuda")
    X[:, 0], W[:, 0] = v, 1
    for act in ACTS:
        check_values(dl.diffuser_linear(X, W, activation=act_code(dl, act)), act, v)
        Y, pre = dl.diffuser_linear(X, W, activation=act_code(dl, act), save_pre=True)
        check_values(Y, act, v)
        assert torch.equal(pre.nan_to_num(1.0), v[:, None].expand(T, F).nan_to_num(1.0))


@pytest.mark.parametrize("kernel", [k for k in sizes.GATED], ids=lambda k: "-".join(map(str, k)))
def test_gated_values_at_limits(dl, kernel):
    T, D, F = max(sizes.GATED[kernel], key=lambda s: s[0])
    finite = [x for x in BEYOND if abs(x) < float("inf")] + TAILS       # (an infinity would make u NaN as well)
    v = spread(finite, T)
    X, W = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(2 * F, D, dtype=torch.bfloat16, device="cuda")
    X[:, 0], X[:, 1], W[:F, 0], W[F:, 1] = v, 1, 1, 1
    for act in ACTS:
        H, pre = dl.diffuser_gated_linear(X, W, activation=act_code(dl, act), save_pre=True)
        check_values(H, act, v)
        assert torch.equal(pre[:, :F], v[:, None].expand(T, F)) and (pre[:, F:] == 1).all()
        check_values(dl.diffuser_gated_linear(X, W, activation=act_code(dl, act)), act, v)
    # a row with an infinity or NaN stays in its row
    X[7 % T, 0] = float("nan")
    bad = dl.diffuser_gated_linear(X, W, activation=dl.DIFFUSER_ACT_SILU)
    H = dl.diffuser_gated_linear(X.nan_to_num(0.5), W, activation=dl.DIFFUSER_ACT_SILU)
    keep = torch.arange(T, device="cuda") != 7 % T
    assert bad[7 % T].isnan().all() and torch.equal(bad[keep], H[keep])


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 70, 300, 5000])
def test_slopes_at_limits(dl, T):
    # through unit gradients and a unit weight; each kernel of the backward has its own slopes
    F = 72
    eye = torch.eye(F, dtype=torch.bfloat16, device="cuda")
    far = [x for x in BEYOND if x == x]
    for act in ACTS:
        for values in (TAILS, far, TAILS[::-1]):
            v = torch.tensor((values * (T * F // len(values) + 1))[:T * F], dtype=torch.bfloat16, device="cuda").view(T, F)
            X, one = draw(1, T, F), torch.ones(T, F, dtype=torch.bfloat16, device="cuda")
            dX, _, db = dl.diffuser_linear_backward(X, eye, one, pre=v, activation=act_code(dl, act), with_dW=False)
            p = v.double()
            s = slope64(act, p)
            beyond = p.abs() > 1e30
            s = torch.where(beyond, (p > 0).double() if act != "none" else torch.ones_like(p), s)
            # near 0 the slopes are sums of two terms of their own size
            tol = REL * s.abs() + (2.0 ** -20 if act != "none" else 0) * (p.abs() < 2) + TINY
            assert ((dX.double() - s).abs() <= tol).all(), (act, T)
            # gated, with u = 1 and weights that keep the gate's half: the same slopes
            pre = torch.cat((v, one), -1)
            W = torch.cat((eye, torch.zeros_like(eye)))
            if not beyond.any():                                 # act(inf) 0 in the other half would be NaN
                dXg, _ = dl.diffuser_gated_linear_backward(X, W, one, pre, activation=act_code(dl, act), with_dW=False)
                assert ((dXg.double() - s).abs() <= tol).all(), (act, T)
                # and the values in the up half's gradient
                dXu, _ = dl.diffuser_gated_linear_backward(X, W.roll(F, 0), one, pre, activation=act_code(dl, act), with_dW=False)
                a = act64(act, p)
                assert ((dXu.double() - a).abs() <= REL * a.abs() + TINY).all(), (act, T)
