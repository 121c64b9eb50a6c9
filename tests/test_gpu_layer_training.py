"""One training step of a transformer layer around the module, all of it by the library's calls
(the heads' concatenation and the permutes of Q, K, V between them are copies of the caller's),
against automatic differentiation of the formulas in 64 bits.

The reference rounds each stored tensor of the forward to bf16 where the library does.  On the way
back every stored gradient is rounded once (U = 2^-8 of its 2-norm at most): output, the gated
product's dH, its dP, its dX, the sum with the residual's, the heads', the module's, the norms'
and the projection's: nine before the input's last sum, in linear maps whose gain on the rounding
noise is that on the gradient itself.  Ten half steps bound each gradient's 2-norm."""
import numpy as np
import pytest

from tests.test_gpu_layer_ops import U, act64, dl, draw, layer_weights, near, norm64, turn64

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
HOPS, ALPHA = 3, 0.1


def train_step(dl, g, P, X, dY, act):
    """The layer's output and the gradients of its input and weights."""
    B, n, D = X.shape
    H = D // 64
    Q, K, V = dl.diffuser_qkv_projection(X, P["qkv"], H)
    q, k = dl.diffuser_qk_norm_rope(Q, K, P["nq"], P["nk"])
    Z = dl.diffuser_forward(q, k, V, g, HOPS, ALPHA)
    heads = Z.transpose(1, 2).reshape(B, n, D)
    A = dl.diffuser_linear(heads, P["o"], bias=P["ob"], residual=X)
    F, pre = dl.diffuser_gated_linear(A, P["gu"], activation=act, save_pre=True)
    Y = dl.diffuser_linear(F, P["down"], residual=A)

    G = {}
    dF, G["down"], _ = dl.diffuser_linear_backward(F, P["down"], dY, with_bias=False)
    dA, G["gu"] = dl.diffuser_gated_linear_backward(A, P["gu"], dF, pre, activation=act)
    dA = dA + dY
    dheads, G["o"], G["ob"] = dl.diffuser_linear_backward(heads, P["o"], dA)
    dZ = dheads.view(B, n, H, 64).transpose(1, 2).contiguous()
    dq, dk, dV = dl.diffuser_backward(q, k, V, dZ, g, HOPS, ALPHA)
    dQ, dK, G["nq"], G["nk"] = dl.diffuser_qk_norm_rope_backward(Q, K, dq, dk, P["nq"], P["nk"])
    dP = torch.stack((dQ, dK, dV)).permute(1, 3, 0, 2, 4).reshape(B, n, 3 * D)
    dX, G["qkv"], _ = dl.diffuser_linear_backward(X, P["qkv"], dP, with_bias=False)
    G["X"] = dX + dA
    return Y, G


class Round(torch.autograd.Function):
    """To bf16 on the way forward, the identity on the way back."""
    @staticmethod
    def forward(ctx, t):
        return t.bfloat16().double()

    @staticmethod
    def backward(ctx, g):
        return g


def reference(g_csr, P, X, dY, act):
    r = Round.apply
    B, n, D = X.shape
    H = D // 64
    w = {k: v.double().requires_grad_(True) for k, v in P.items()}
    x = X.double().requires_grad_(True)
    q, k, v = r(x @ w["qkv"].T).view(B, n, 3, H, 64).permute(2, 0, 3, 1, 4)
    pos = torch.arange(n, device="cuda").expand(B, n)
    q, k = (r(turn64(norm64(t, w[m], 1e-6), pos, 64, False, 10000.0)) for t, m in ((q, "nq"), (k, "nk")))
    row_ptr, col = g_csr
    mask = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        mask[i, torch.from_numpy(col[row_ptr[i]:row_ptr[i + 1]].astype(np.int64))] = True
    a = torch.softmax((q @ k.transpose(-1, -2) / 8).masked_fill(~mask.cuda(), float("-inf")), -1)
    z = v
    for _ in range(HOPS):
        z = (1 - ALPHA) * (a @ z) + ALPHA * v
    A = r(x + r(z).transpose(1, 2).reshape(B, n, D) @ w["o"].T + w["ob"])
    gate, up = (A @ w["gu"].T).chunk(2, -1)
    y = A + r(act64(act, gate) * up) @ w["down"].T
    names = list(w)
    grads = torch.autograd.grad(y, [x] + [w[k] for k in names], dY.double())
    return y.detach(), dict(zip(["X"] + names, grads))


@pytest.mark.parametrize("size", [(2, 300, 128, 344), (1, 517, 192, 520), (1, 3, 64, 72)], ids=str)
def test_a_layer_trains(dl, size):
    B, n, D, F = size
    g = dl.diffuser_build_graph(n, 16, min(3, n), rand_per_row=5, seed=0)
    P, X, dY = layer_weights(D, F), draw(40, B, n, D), draw(41, B, n, D)
    Y, G = train_step(dl, g, P, X, dY, dl.DIFFUSER_ACT_SILU)
    ref, want = reference(dl.diffuser_graph_copy_csr(g), P, X, dY, "silu")
    near(Y, ref, "layer", limit=8 * U)
    assert set(G) == set(want)
    for name in want:
        assert G[name].shape == want[name].shape
        near(G[name], want[name], name, limit=10 * U)


def test_a_captured_step(dl):
    # the whole step in a graph, replayed on new inputs, gives the eager step's bits
    B, n, D, F = 1, 300, 128, 344
    g = dl.diffuser_build_graph(n, 16, 3, rand_per_row=5, seed=0)
    P = layer_weights(D, F)
    X, dY = draw(40, B, n, D), draw(41, B, n, D)
    train_step(dl, g, P, X, dY, dl.DIFFUSER_ACT_SILU)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        Y, G = train_step(dl, g, P, X, dY, dl.DIFFUSER_ACT_SILU)
    X.copy_(draw(50, B, n, D))
    dY.copy_(draw(51, B, n, D))
    gr.replay()
    torch.cuda.synchronize()
    y, h = train_step(dl, g, P, X, dY, dl.DIFFUSER_ACT_SILU)
    assert torch.equal(Y, y)
    for name in h:
        assert torch.equal(G[name], h[name]), name
