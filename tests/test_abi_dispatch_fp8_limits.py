"""Host-side checks at the largest sizes of the dispatch and FP8 ragged entry points (no GPU needed)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def L():
    from fp8_block_scaled_grouped_amd import moe355
    if not os.path.exists(moe355.LIB_PATH):
        pytest.skip("libmoe355.so not built")
    return moe355.lib()


P = ctypes.c_void_p(16)
MOST = 2 ** 31 - 1


def test_rows_whose_tiles_pass_32_bits_are_refused(L):
    """The kernels count a segment's tiles as (rows + 255) / 256 and its blocks as (rows + 127) / 128 in 32 bits."""
    for R in (MOST - 254, MOST):
        assert L.grouped_gemm_fp8(P, P, 16, 1, 1, P, P, 1, P, R, 1, 8, 16, P, 8, 0, None) == -2
        assert L.grouped_gemm_fp8_wgrad(P, P, P, P, P, R, 1, 8, 8, P, 0, None) == -2


def test_rows_whose_elements_pass_32_bits_are_refused(L):
    """moe_combine_grad steps 256 elements of a row that starts off 16 bytes at a time in 32 bits."""
    for H in (MOST - 254, MOST):
        assert L.moe_combine_grad(P, H, P, H, 0, 1, H, 1, P, 1, P, 1, P, H, P, None) == -2
