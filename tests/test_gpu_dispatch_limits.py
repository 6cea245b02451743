"""Dispatch and combine: what autograd keeps, and the largest sizes; oracles and tolerances as in test_gpu_dispatch.py."""
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


# ------------------------------------------------------------------ many pairs
def _sorted(ids, E):
    """The oracle's order by torch's stable sort (its own loop is long)."""
    flat = ids.reshape(-1).long()
    key, order = torch.sort(torch.where((flat >= 0) & (flat < E), flat, E), stable=True)
    off, n = torch.searchsorted(key, torch.arange(E + 1)), int((key < E).sum())
    rop = torch.full((flat.numel(),), -1)
    rop[order[:n]] = torch.arange(n)
    return off, rop.view(ids.shape), torch.where(key < E, order, -1)


# chunks are of 4096 pairs up to 256 of them; past 1048576 pairs of 8192 and more, whose waves hold 256 ids in registers and read the others
# twice: parts of 512, 768 (the last ones cut short) and 512 with all experts that there may be
@pytest.mark.parametrize("T,k,E", [(131072, 8, 256), (131073, 8, 256), (300001, 8, 256), (150011, 7, 1024), (1100000, 1, 3)])
def test_group_of_more_than_a_million_pairs(m, T, k, E):
    print("group", T, k, E, flush=True)
    ids = _ids(T, k, E, T)
    ref = _sorted(ids, E)
    wide = torch.full((T, k + 3), 77, dtype=torch.int32)      # rows with a stride
    wide[:, :k] = ids
    for x in (ids.to(DEV), wide.to(DEV)[:, :k]):
        for got, want in zip(m.moe_group(x, E), ref):
            assert torch.equal(got.cpu().long(), want)


@pytest.mark.parametrize("T,k,E", [(140000, 8, 16)])
def test_group_of_more_than_a_million_pairs_on_one_expert_and_on_none(m, T, k, E):
    one = torch.full((T, k), E - 1, dtype=torch.int32, device=DEV)
    o, r, p = m.moe_group(one, E)
    assert o.tolist() == [0] * E + [T * k] and torch.equal(r.flatten(), torch.arange(T * k, device=DEV, dtype=torch.int32))
    assert torch.equal(p, r.flatten())
    o, r, p = m.moe_group(torch.full_like(one, E), E)
    assert o.tolist() == [0] * (E + 1) and (r == -1).all() and (p == -1).all()


def test_gradients_of_rows_past_two_to_the_31_bytes(m):
    """The last rows of two buffers of 4.3 GB: gradients of rows and weights.  Multiples of 1/4 up to 2 (rows) and 1 (dout), so a product is a
    multiple of 1/16 and sums of H = 2^15 of them, below 2^16, are exact in fp32 in any order."""
    T, k, H = 4, 2, 1 << 15
    R = (1 << 32) // (2 * H) + 64
    rows, drows = (torch.zeros((R, H), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    rop = torch.tensor([[R - 1, 0], [R - 2, 1], [R // 2, R // 2 + 1], [R - 64, 7]], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(1)
    y = torch.randint(-8, 9, (T, k, H), generator=g).to(DEV) / 4
    dout = torch.randint(-4, 5, (T, H), generator=g).to(DEV) / 4
    rows[rop.long()] = y.to(torch.bfloat16)
    w = torch.tensor([[0.5, 1.0], [2.0, 0.25], [1.0, 4.0], [0.125, 8.0]], device=DEV)
    d, dw = m.moe_combine_grad(dout.to(torch.bfloat16), rows, rop, w, drows)
    assert d is drows and torch.equal(dw, (y * dout[:, None]).sum(-1))
    assert torch.equal(drows[rop.long()], (w[..., None] * dout[:, None]).to(torch.bfloat16))
    rest = torch.ones(R, dtype=torch.bool, device=DEV)
    rest[rop.long().flatten()] = False
    assert not drows.any(1)[rest].any()
