"""Which of its two kernels the attention over chosen blocks takes, seen on the workspace it asks for: none
by query, the lists and partial sums by block."""
import ctypes

import pytest

from sparse_long_sequence_gb300 import build as cuda_build


@pytest.fixture(scope="module")
def size():
    lib = ctypes.CDLL(cuda_build.build())
    f = lib.diffuser_selected_attention_workspace_size
    f.argtypes = [ctypes.c_int64] * 5 + [ctypes.c_int32] * 2 + [ctypes.c_void_p]

    def call(B, Hq, Hk, n, m, top):
        b = ctypes.c_size_t()
        assert f(B, Hq, Hk, n, m, 64, top, ctypes.addressof(b)) == 0
        return b.value
    return call


@pytest.mark.parametrize("Hq,Hk", [(8, 8), (32, 8), (64, 8), (64, 4)])
@pytest.mark.parametrize("top", [1, 16, 64])
@pytest.mark.parametrize("m", [4096, 65536, 1 << 20])
def test_single_tokens_take_no_workspace(size, Hq, Hk, top, m):
    """However many sequences: no key block has two of their queries."""
    for B in (1, 16, 64, 81, 256, 1024):
        assert size(B, Hq, Hk, 1, m, top) == 0


@pytest.mark.parametrize("B,Hq,Hk,n,m,top", [
    (16, 32, 8, 2, 16384, 16), (64, 32, 8, 8, 16384, 16), (1, 4, 1, 256, 4096, 16), (16, 32, 8, 32, 16384, 16),
    (1, 2, 2, 5120, 0, 16), (0, 32, 8, 100, 4096, 16), (64, 32, 8, 0, 4096, 16)])
def test_queries_that_hardly_meet(size, B, Hq, Hk, n, m, top):
    assert size(B, Hq, Hk, n, m, top) == 0


@pytest.mark.parametrize("B,Hq,Hk,n,m,top", [
    (64, 32, 8, 32, 4096, 16), (1, 1, 1, 1024, 1024, 16), (1, 12, 12, 256, 256, 4), (2, 4, 2, 5120, 5120, 1),
    (1, 16, 16, 16384, 16384, 16), (4, 4096, 4, 1, 16384, 16)])
def test_queries_that_share_blocks(size, B, Hq, Hk, n, m, top):
    assert size(B, Hq, Hk, n, m, top) > 0
