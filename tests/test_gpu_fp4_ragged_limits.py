"""4-bit and ragged products at the ends of what their calls take."""
import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def m():
    import fp8_block_scaled_grouped_amd as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("first", [2 ** 31 - 209, 2 ** 31 - 70000])
def test_segment_that_ends_near_2_to_31(m, first):
    # rows from `first` up to 2^31 - 8: the row numbers of later passes would leave 32 bits
    torch.cuda.empty_cache()
    R, N, K = 2 ** 31 - 8, 1, 32
    if torch.cuda.mem_get_info()[0] < 150 * 2 ** 30:
        pytest.skip("needs 142 GB for %d rows" % R)
    rng = np.random.default_rng(1)
    q, s = fp4.quant_groups(rng.normal(0, 0.02, (N, K)).astype(np.float32), 32, True)
    w = fp4.dequant_groups(q, s, 32)
    x, c = torch.empty((R, K), dtype=torch.bfloat16, device=DEV), torch.empty((R, N), dtype=torch.bfloat16, device=DEV)
    rows = R - first
    x[first:] = torch.randn((rows, K), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    c[first - 4096:] = 7.0
    print("rows near 2^31", first, flush=True)
    m.grouped_gemm_fp4(x, torch.tensor(q, device=DEV)[None], torch.tensor(s, device=DEV)[None],
                       torch.tensor([first, R], dtype=torch.int32, device=DEV), 32, c)
    xf = x[first:].double().cpu().numpy()
    d = (K + 8) * 2.0 ** -23 * (np.abs(xf) @ np.abs(w).T)
    lo, hi = (torch.tensor(v).to(torch.bfloat16).double().numpy() for v in (xf @ w.T - d, xf @ w.T + d))
    got = c[first:].double().cpu().numpy()
    assert ((got >= lo) & (got <= hi)).all()
    assert bool((c[first - 4096:first] == 7).all())
    del x, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradient_that_starts_off_16_bytes(m, dtype):
    # the backward of a concatenation hands grouped_linear a view of its gradient that starts 6 bytes in
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randn(s, generator=g).to(dtype).to(DEV) for s in ((6, 16), (2, 24, 16)))
    od, up = torch.tensor([0, 2, 6], dtype=torch.int32, device=DEV), torch.randn(6 * 24 + 3, generator=g).to(dtype).to(DEV)
    tx, tw, head = x.clone().requires_grad_(), w.clone().requires_grad_(), torch.zeros(3, dtype=dtype, device=DEV, requires_grad=True)
    torch.cat([head, m.grouped_linear(tx, tw, od).flatten()]).backward(up)
    dy = up[3:].clone().view(6, 24)
    assert torch.equal(tx.grad, m.grouped_gemm_dgrad(dy, w, od)) and torch.equal(tw.grad, m.grouped_gemm_wgrad(dy, x, od))
