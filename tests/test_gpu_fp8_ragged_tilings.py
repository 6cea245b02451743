"""Every tile of the FP8 expert products against the 64-bit oracle, with several tiles a workgroup; tolerances as in test_gpu_fp8_ragged.py."""
import numpy as np
import pytest
import torch

from oracle import fp8_ragged as o
from tests import fp8_ragged_tilings as t
from tests.test_gpu_fp8_ragged import DEV, DT, _check_wgrad, _dev, _f64, _offsets, _operands, _randn, _wide_range

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import fp8_block_scaled_grouped_amd as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("fmt", ["e8m0", "fp32"])
@pytest.mark.parametrize("counts,N,K", t.PRODUCTS)
def test_product(m, counts, N, K, fmt):
    print("grouped_gemm_fp8", counts[:4], len(counts), N, K, fmt, flush=True)
    ops = _operands(counts, len(counts), N, K, fmt, N + K)
    dtype = "fp16" if K % 32 else "bf16"
    base = torch.full((ops.R + 2, N), 7.0, dtype=DT[dtype], device=DEV)
    y = m.grouped_gemm_fp8(*ops.dev, _dev(ops.off), base[1:-1])
    ops.check(y, dtype, "y")
    assert (base[0] == 7).all() and (base[-1] == 7).all()


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("counts,N,K", t.GRADIENTS)
def test_wgrad(m, counts, N, K, out):
    print("grouped_gemm_fp8_wgrad", counts[:4], len(counts), N, K, out, flush=True)
    off, E = _offsets(counts), len(counts)
    R = off[-1]
    dy, x = _wide_range((R, N), "fp16", 1), _randn((R, K), "fp16", 2)
    dyt, dys, used = o.quant_columns(_f64(dy), off)
    xt, xs, _ = o.quant_columns(_f64(x), off)
    for a, fill in ((dyt, 0x7f), (xt, 0x7f), (dys, 255), (xs, 255)):       # blocks that no expert has are not read
        a[~used] = fill
    base = torch.full((E * N * K + 256,), 7.0, dtype=DT[out], device=DEV)
    dw = base[128:-128].view(E, N, K)
    m.grouped_gemm_fp8_wgrad(*(torch.tensor(a, device=DEV) for a in (dyt, dys, xt, xs)), _dev(off), R, dw)
    _check_wgrad(dw, dyt, dys, xt, xs, off, max(counts), out)
    assert (dw[np.array(counts) == 0] == 0).all() and (base[:128] == 7).all() and (base[-128:] == 7).all()
