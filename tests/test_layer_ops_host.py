"""Host-side refusals of the operators around the module: every argument check answers
before anything touches a device (no compute call is made here)."""
import ctypes

import pytest

from sparse_long_sequence_gb300 import build as cuda_build

OK, INVALID, UNSUPPORTED, OVERFLOW, WORKSPACE = 0, 1, 2, 3, 7
vp, i32, i64, f32, f64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                              ctypes.c_size_t)
A = [0x10000000 * (k + 1) for k in range(12)]      # addresses that nothing reads


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(cuda_build.build())
    sig = {
        "diffuser_qk_norm_rope": [vp, vp, i32, i64, i64, i64, i64, i32, vp, vp, f32, f64, i32, i32, vp, i64, vp, vp, vp],
        "diffuser_qk_norm_rope_backward_workspace_size": [i64, i64, i64, i64, i32, vp],
        "diffuser_qk_norm_rope_backward": [vp, vp, vp, vp, i32, i64, i64, i64, i64, i32, vp, vp, f32, f64, i32, i32, vp,
                                           i64, vp, vp, vp, vp, vp, sz, vp],
        "diffuser_linear": [vp, vp, vp, vp, i64, i32, i32, i32, vp, vp, vp],
        "diffuser_linear_backward_workspace_size": [i64, i32, i32, i32, vp],
        "diffuser_linear_backward": [vp, vp, vp, vp, i64, i32, i32, i32, vp, vp, vp, vp, sz, vp],
        "diffuser_gated_linear": [vp, vp, i64, i32, i32, i32, vp, vp, vp],
        "diffuser_gated_linear_backward_workspace_size": [i64, i32, i32, vp],
        "diffuser_gated_linear_backward": [vp, vp, vp, vp, i64, i32, i32, i32, vp, vp, vp, sz, vp],
    }
    for name, args in sig.items():
        getattr(lib, name).argtypes = args
    return lib


QK = dict(Q=A[0], K=A[1], dtype=1, B=1, Hq=2, Hk=2, n=4, d=64, wq=A[2], wk=A[3], eps=1e-6, theta=1e4, rot=64, inter=0,
          pos=None, off=0, Qo=A[4], Ko=A[5])


@pytest.mark.parametrize("change,status", [
    (dict(d=128), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=80), INVALID),
    (dict(rot=-16), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(theta=0.5), INVALID), (dict(theta=float("nan")), INVALID), (dict(theta=float("inf")), INVALID),
    (dict(B=-1), INVALID), (dict(n=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=5000), INVALID),
    (dict(B=1 << 31), INVALID), (dict(B=1 << 30, n=1 << 30), OVERFLOW),
    (dict(Q=None), INVALID), (dict(K=None), INVALID), (dict(Qo=None), INVALID), (dict(Ko=A[5] + 2), INVALID),
    (dict(wq=A[2] + 8), INVALID), (dict(pos=A[6] + 4), INVALID), (dict(Qo=A[0] + 16), INVALID), (dict(Qo=A[1]), INVALID),
    (dict(Ko=A[4]), INVALID), (dict(Qo=A[2]), INVALID), (dict(pos=A[4]), INVALID)])
def test_qk_refusals(lib, change, status):
    c = dict(QK, **change)
    assert lib.diffuser_qk_norm_rope(*[c[k] for k in QK], None) == status


def test_qk_of_no_tokens(lib):
    for change in (dict(n=0), dict(B=0)):
        c = dict(QK, Q=None, K=None, Qo=None, Ko=None, **change)
        assert lib.diffuser_qk_norm_rope(*[c[k] for k in QK], None) == OK


QKB = dict(Q=A[0], K=A[1], dQo=A[2], dKo=A[3], dtype=1, B=1, Hq=2, Hk=2, n=4, d=64, wq=A[4], wk=A[5], eps=1e-6, theta=1e4,
           rot=64, inter=0, pos=None, off=0, dQ=A[6], dK=A[7], dwq=A[8], dwk=A[9], ws=A[10], bytes=1 << 20)


@pytest.mark.parametrize("change,status", [
    (dict(wq=None), INVALID), (dict(wk=None), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=A[10] + 64), WORKSPACE),
    (dict(bytes=64), WORKSPACE), (dict(dQ=A[0]), INVALID), (dict(dQ=A[2]), INVALID), (dict(dK=A[6]), INVALID),
    (dict(dwq=A[8] + 2), INVALID), (dict(dwk=A[8]), INVALID), (dict(ws=A[0]), INVALID), (dict(dQo=None), INVALID),
    (dict(dKo=A[3] + 8), INVALID), (dict(ws=A[6]), INVALID)])
def test_qk_backward_refusals(lib, change, status):
    c = dict(QKB, **change)
    assert lib.diffuser_qk_norm_rope_backward(*[c[k] for k in QKB], None) == status


LIN = dict(X=A[0], W=A[1], bias=A[2], res=A[3], T=5, D=64, F=72, act=0, Y=A[4], pre=A[5])
SIZES = [(dict(T=-1), INVALID), (dict(T=(1 << 30) + 1), INVALID), (dict(D=0), INVALID), (dict(F=0), INVALID),
         (dict(D=-8), INVALID), (dict(D=12), UNSUPPORTED), (dict(F=76), UNSUPPORTED), (dict(D=65544), UNSUPPORTED),
         (dict(F=65544), UNSUPPORTED), (dict(act=5), UNSUPPORTED), (dict(act=-1), UNSUPPORTED), (dict(X=None), INVALID),
         (dict(W=None), INVALID), (dict(X=A[0] + 8), INVALID), (dict(W=A[1] + 2), INVALID)]


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(Y=None), INVALID), (dict(Y=A[0]), INVALID), (dict(Y=A[3] + 16), INVALID), (dict(Y=A[2]), INVALID),
    (dict(pre=A[4]), INVALID), (dict(pre=A[3]), INVALID), (dict(pre=A[5] + 2), INVALID), (dict(bias=A[2] + 2), INVALID),
    (dict(res=A[3] + 2), INVALID)])
def test_linear_refusals(lib, change, status):
    c = dict(LIN, **change)
    assert lib.diffuser_linear(*[c[k] for k in LIN], None) == status


LINB = dict(X=A[0], W=A[1], dY=A[2], pre=A[3], T=5, D=64, F=72, act=4, dX=A[4], dW=A[5], db=A[6], ws=A[7], bytes=1 << 20)


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(pre=None), INVALID), (dict(dY=None), INVALID), (dict(dX=A[0]), INVALID), (dict(dW=A[1]), INVALID),
    (dict(dX=A[2]), INVALID), (dict(dW=A[4]), INVALID), (dict(db=A[6] + 2), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=A[7] + 16), WORKSPACE), (dict(bytes=100), WORKSPACE), (dict(ws=A[2]), INVALID), (dict(ws=A[4]), INVALID)])
def test_linear_backward_refusals(lib, change, status):
    c = dict(LINB, **change)
    assert lib.diffuser_linear_backward(*[c[k] for k in LINB], None) == status


GAT = dict(X=A[0], W=A[1], T=5, D=64, F=72, act=4, H=A[2], pre=A[3])


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(H=None), INVALID), (dict(H=A[0]), INVALID), (dict(pre=A[2]), INVALID), (dict(pre=A[1] + 64), INVALID)])
def test_gated_refusals(lib, change, status):
    c = dict(GAT, **change)
    assert lib.diffuser_gated_linear(*[c[k] for k in GAT], None) == status


GATB = dict(X=A[0], W=A[1], dH=A[2], pre=A[3], T=5, D=64, F=72, act=4, dX=A[4], dW=A[5], ws=A[6], bytes=1 << 20)


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(pre=None), INVALID), (dict(dH=None), INVALID), (dict(dX=A[3]), INVALID), (dict(dW=A[4]), INVALID),
    (dict(ws=None), WORKSPACE), (dict(bytes=100), WORKSPACE), (dict(ws=A[3]), INVALID)])
def test_gated_backward_refusals(lib, change, status):
    c = dict(GATB, **change)
    assert lib.diffuser_gated_linear_backward(*[c[k] for k in GATB], None) == status


def test_products_of_no_tokens(lib):
    assert lib.diffuser_linear(None, A[1], None, None, 0, 64, 72, 0, None, None, None) == OK
    assert lib.diffuser_gated_linear(None, A[1], 0, 64, 72, 4, None, None, None) == OK


def test_workspace_sizes(lib):
    b = ctypes.c_size_t()
    for T in (0, 1, 5, 8192, 1 << 30):
        for act in (0, 4):
            assert lib.diffuser_linear_backward_workspace_size(T, 64, 72, act, ctypes.byref(b)) == OK
            assert b.value % 256 == 0 and b.value >= (0 if T <= 4 else T * 72 * 2 if act else 1)
        assert lib.diffuser_gated_linear_backward_workspace_size(T, 64, 72, ctypes.byref(b)) == OK
        assert b.value % 256 == 0 and b.value >= (0 if T <= 4 else T * 72 * 4)
    for n in (0, 1, 1 << 20):
        assert lib.diffuser_qk_norm_rope_backward_workspace_size(2, 3, 4, n, 64, ctypes.byref(b)) == OK
        assert 0 < b.value <= 152 * 4 * 512
    assert lib.diffuser_linear_backward_workspace_size(5, 64, 72, 0, None) == INVALID
    assert lib.diffuser_gated_linear_backward_workspace_size(5, 60, 72, ctypes.byref(b)) == UNSUPPORTED
