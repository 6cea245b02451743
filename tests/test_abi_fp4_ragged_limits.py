"""Host-side limits of the 4-bit products: sizes past what a launch takes give the documented code before anything is
launched (no GPU needed)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def L():
    from fp8_block_scaled_grouped_amd import moe355
    if not os.path.exists(moe355.LIB_PATH):
        pytest.skip("libmoe355.so not built")
    return moe355.lib()


@pytest.mark.parametrize("M", [1, 8, 16, 32, 64])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("fp16", [0, 1])
@pytest.mark.parametrize("e8m0", [0, 1])
def test_more_columns_than_a_launch_has_threads(L, M, group, fp16, e8m0):
    p, N = ctypes.c_void_p(16), 2 ** 31 - 1
    assert L.gemm_fp4_groupscale(p, fp16, 32, p, p, e8m0, group, M, N, 32, p, N, None, 0, None) == -2
    assert L.grouped_gemm_fp4(p, fp16, 32, p, p, e8m0, group, p, M, 1, N, 32, p, N, None) == -2
