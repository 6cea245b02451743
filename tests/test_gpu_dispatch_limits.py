"""Dispatch and combine: what autograd keeps, and the largest sizes; oracles and tolerances as in test_gpu_dispatch.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_dispatch import DEV, _ids, _place, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import fp8_block_scaled_grouped_amd as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("T,k,H", [(20, 3, 48), (7, 2, 33)])
def test_rows_are_kept_for_the_gradient_of_the_weights_alone(m, T, k, H):
    """With weights that need no gradient (a router's choice) the gradient of the rows is weights * dout: the rows are neither held nor
    have to stay as they were."""
    _, rop, n = _place(T, k, 6, 5, outside=False)
    leaf = _randn((T * k, H), "fp32", 1).to(DEV).requires_grad_()
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(2)).to(DEV)
    dout = _randn((T, H), "fp32", 3).to(DEV)
    rows = leaf * 1.0
    out = m.moe_combine(rows, rop, w)
    keep = out.detach().clone()
    assert all(s is None or s.shape != rows.shape for s in out.grad_fn.saved_tensors)
    with torch.no_grad():
        rows.zero_()
    (d,) = torch.autograd.grad(out, leaf, dout)
    ref = torch.zeros_like(leaf)
    ref[rop.long().flatten()] = (w[..., None] * dout[:, None]).reshape(T * k, H)
    assert torch.equal(d, ref) and torch.equal(out, keep)
    # with a gradient of the weights they are, and a change is refused
    w.requires_grad_()
    rows = leaf * 1.0
    out = m.moe_combine(rows, rop, w)
    dl, dw = torch.autograd.grad(out, (leaf, w), dout, retain_graph=True)
    assert torch.equal(dl, ref) and dw.shape == w.shape
    assert torch.equal(torch.autograd.grad(out, w, dout, retain_graph=True)[0], dw)
    with torch.no_grad():
        rows.zero_()
    with pytest.raises(RuntimeError):
        torch.autograd.grad(out, (leaf, w), dout)
