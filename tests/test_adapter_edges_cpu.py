"""Refusals of the adapters' gradients at the largest sizes (fake pointers,
never dereferenced)."""
import pytest

A = 0x10000
OK, NULL, SHAPE, ARG = 0, 1, 2, 5


@pytest.fixture(scope="module")
def w8():
    import w8a8_int8_quantized_token_amd as pkg
    return pkg


def call(w8, M, N, K, R, L, dx=A, da=A, db=A, ws=A, n=1 << 50):
    return w8.lib.w8a8_linear_adapters_backward(A, A, A, A, A, A, A, A, A, dx, da, db, M, N, K, R, L, ws, n, None)


@pytest.mark.parametrize("M,N,K,R,L", [(65, 8192, 8192, 8, 65536), (65, 16384, 64, 8, 65536), (65, 64, 16384, 8, 65536),
                                       (65, 8192, 16384, 128, 32768)])
def test_more_matrices_than_a_launch_lays_out(w8, M, N, K, R, L):
    size = w8.lib.w8a8_linear_adapters_backward_workspace
    assert call(w8, M, N, K, R, L) == SHAPE and size(M, N, K, R, L, 1, 1, 1) == 0
    assert call(w8, M, N, K, R, L, da=None, db=None) == SHAPE and size(M, N, K, R, L, 1, 0, 0) == 0
    half = L // 4
    assert call(w8, M, N, K, R, half, ws=None) == NULL and size(M, N, K, R, half, 1, 1, 1) > 0
    # b's gradient alone needs none of them
    assert call(w8, M, N, K, R, half, dx=None, da=None, n=16) == ARG and size(M, N, K, R, half, 0, 0, 1) > 0


def test_what_needs_no_layout_is_taken(w8):
    size = w8.lib.w8a8_linear_adapters_backward_workspace
    M, N, K, R, L = 4, 8192, 8192, 8, 65536
    assert call(w8, M, N, K, R, L, dx=None, da=None, n=16) == ARG and size(M, N, K, R, L, 0, 0, 1) > 0
    assert call(w8, M, N, K, R, L, dx=None, n=16) == ARG and size(M, N, K, R, L, 0, 1, 1) > 0


def test_larger_ranks_of_as_many_adapters(w8):
    """Ranks above 48 take more workgroups, and more than one dimension of a grid has threads for."""
    size = w8.lib.w8a8_linear_adapters_backward_workspace
    for R in (8, 48, 64, 128):
        assert call(w8, 4, 8192, 1024, R, 65536, dx=None, da=None, n=16) == ARG and size(4, 8192, 1024, R, 65536, 0, 0, 1) > 0, R
