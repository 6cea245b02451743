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


def test_sizes_that_32_bits_would_cut_are_refused(L):
    """The library's sizes are C ints: a tensor of 2^32 + n rows must not pass for one of n (on tensors without memory)."""
    import torch

    import fp8_block_scaled_grouped_amd as m
    big = 2 ** 32 + 16
    e = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="meta")
    i, u = torch.int32, torch.uint8
    few, x, rop = e(4, 2, dtype=i), e(4, 16), e(big, 2, dtype=i)
    w8, ws, off = e(2, 16, 16, dtype=u), e(2, 1, 1, dtype=torch.float32), e(3, dtype=i)
    for call in (lambda: m.moe_group(rop, 4), lambda: m.moe_group(e(4, big, dtype=i), 4), lambda: m.moe_group(few, 2 ** 32 + 4),
                 lambda: m.moe_group_workspace(big, 2, 4), lambda: m.moe_group_workspace(4, 2, 2 ** 32 + 4),
                 lambda: m.moe_dispatch(e(big, 16), rop), lambda: m.moe_dispatch(e(4, big), few), lambda: m.moe_dispatch(x, few, e(big, 16)),
                 lambda: m.moe_dispatch(e(1 << 26, 8), e(1 << 26, 64, dtype=i)),
                 lambda: m.moe_combine(e(big, 16), few), lambda: m.moe_combine(e(8, big), few), lambda: m.moe_combine(e(8, 16), rop),
                 lambda: m.moe_combine_grad(x, e(big, 16), few, e(4, 2, dtype=torch.float32)),
                 lambda: m.fp8_ragged_blocks(big, 2), lambda: m.fp8_ragged_blocks(16, big),
                 lambda: m.grouped_gemm_fp8(e(big, 16, dtype=u), e(big, 1, dtype=torch.float32), w8, ws, off),
                 lambda: m.grouped_gemm_fp8(e(4, 16, dtype=u), e(4, 1, dtype=torch.float32), e(2, big, 16, dtype=u), ws, off)):
        with pytest.raises(ValueError, match=r"below 2\^31"):
            call()
