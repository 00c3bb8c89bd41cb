"""What the MX4 calls ask for, and refuse at the edges of their limits, without a GPU."""
import ctypes

import pytest
import torch

from lossless_bit_weight_amd import mx4

A = ctypes.c_void_p(4096)       # never dereferenced: every call here fails validation


@pytest.mark.parametrize("B,R,K,ldy,ldb", [
    (2, 16, 64, 64, 512),           # the second starts inside the first
    (3, 4, 64, 128, 64),            # room between rows for one more matrix, not for two
    (2, 4, 64, 96, 64), (2, 4, 64, 128, 32),
    (2, 1 << 30, 64, 1 << 39, 32)])  # rows times stride past 2^63
def test_dequantize_refuses_matrices_that_overlap(B, R, K, ldy, ldb):
    assert mx4.lib().mx4_dequantize(A, A, B, R, K, A, 0, ldy, ldb, None) == -2


def test_dequantize_of_zero_rows_needs_no_strides():
    assert mx4.lib().mx4_dequantize(None, None, 3, 0, 64, None, 0, 64, 0, None) == 0


@pytest.mark.parametrize("M,ldx,status", [(1 << 20, 1 << 23, -2), (1 << 24, 1 << 23, -2)])
def test_gemm_refuses_many_rows_far_apart(M, ldx, status):
    """Rows 2^23 elements apart and more go to the few-row kernel, up to 16 * 65535 of them."""
    assert mx4.lib().mx4_gemm(A, M, ldx, A, A, 32, 64, A, 32, 0, None, 0, None) == status


@pytest.mark.parametrize("T,H,I,E,k", [(1, 5120, 1280, 64, 6), (2, 2048, 768, 128, 8)])
def test_moe_workspace_of_tokens_one_by_one(T, H, I, E, k):
    """Tokens that go one by one need their pairs' words and hidden values, no outputs of
    pairs and no places."""
    for dtype, size in ((torch.bfloat16, 4), (torch.float32, 6)):
        need = mx4.mx4_moe_workspace_bytes(T, H, I, E, k, dtype)
        assert T * k * (I * size + 16) <= need <= T * k * (I * size + 128) + 256


@pytest.mark.parametrize("x_mx4", [False, True])
def test_gemm_that_splits_k_refuses_a_bad_workspace(x_mx4):
    M, N, K = 33, 512, 17408
    need = mx4.mx4_gemm_workspace_bytes(M, N, K, x_mx4)
    assert need >= 2 * M * N * 4                # two slices' sums at least
    L = mx4.lib()
    for ws, n in ((None, need), (A, need - 1), (A, 0), (ctypes.c_void_p(4096 + 16), need)):
        if x_mx4:
            rc = L.mx4_gemm_mx4(A, A, M, A, A, N, K, A, N, 0, ws, n, None)
        else:
            rc = L.mx4_gemm(A, M, K, A, A, N, K, A, N, 0, ws, n, None)
        assert rc == -8
