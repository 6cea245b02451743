"""Tokens to their experts, through two FP8 products and back, as a training step runs them.

Exact: the weights have four entries of -1 or 1 in each row and column, tokens are -1, 0 or 1, routing weights 1 or 2, so with at
most 32 rows an expert every value on the way is a whole number that its type holds: y1 <= 4, h <= 4, y2 <= 16, out <= 3 * 2 * 16; dy <= 2,
dh <= 4 * 2, dx <= 3 * 4 * 8; dw2 <= 32 * 2 * 4, dw1 <= 32 * 8 (bf16 holds up to 256, e4m3 up to 16), and a block's scale is a
power of two.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E, K = 6, 48


@pytest.fixture(scope="module")
def m():
    import fp8_block_scaled_grouped_amd as mod
    mod.lib()
    return mod


def _weights(seed):
    """[E, K, K], rows and columns with four entries of -1 or 1."""
    g = torch.Generator().manual_seed(seed)
    n, k = torch.arange(K)[:, None], torch.arange(K)[None, :]
    hit = torch.isin((k - n) % K, torch.tensor([0, 5, 17, 30]))
    return torch.where(hit, torch.randint(0, 2, (E, K, K), generator=g) * 2.0 - 1.0, 0.0)


def _inputs(T, k, seed, outside):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    if outside:
        ids[torch.rand((T, k), generator=g) < 0.3] = -1
    assert torch.bincount(ids[ids >= 0].long(), minlength=E).max() <= 32
    x = torch.randint(-1, 2, (T, K), generator=g).double()
    w = torch.randint(1, 3, (T, k), generator=g).double()
    return ids, x, w, torch.randint(-1, 2, (T, K), generator=g).double()


def _path(m, x, ids, w1, w2, weights):
    offsets, row_of_pair, _ = m.moe_group(ids, E)
    rows = m.moe_dispatch(x, row_of_pair)
    h = torch.relu(m.grouped_linear_fp8(rows, w1, offsets))
    return m.moe_combine(m.grouped_linear_fp8(h, w2, offsets), row_of_pair, weights)


def _plain(x, ids, w1, w2, weights):
    out = torch.zeros_like(x)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y = torch.relu(x[t] @ w1[e].t()) @ w2[e].t()
        out = out.index_add(0, t, weights[t, j, None] * y)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,k,outside", [(1, 1, False), (24, 3, False), (40, 3, True), (7, 2, True)])
def test_path_and_gradients(m, T, k, outside, dtype):
    ids, x, weights, dout = _inputs(T, k, T + k, outside)
    leaves = [t.requires_grad_() for t in (x, _weights(1).double(), _weights(2).double(), weights)]
    ref = _plain(x, ids, *leaves[1:])
    grads = torch.autograd.grad(ref, leaves, dout)
    dev = [t.detach().to(DEV, torch.float32 if i == 3 else dtype).requires_grad_() for i, t in enumerate(leaves)]
    out = _path(m, dev[0], ids.to(DEV), *dev[1:])
    assert torch.equal(out.detach().cpu().double(), ref.detach())
    got = torch.autograd.grad(out, dev, dout.to(DEV, dtype))
    for name, a, b in zip(("dx", "dw1", "dw2", "dweights"), got, grads):
        assert torch.equal(a.cpu().double(), b), name


def test_path_without_any_pair(m):
    """Every expert is held elsewhere: zeros, and zero gradients."""
    ids = torch.full((5, 2), -1, dtype=torch.int32, device=DEV)
    x = torch.ones((5, K), dtype=torch.bfloat16, device=DEV, requires_grad=True)
    w1, w2 = (_weights(i).to(DEV, torch.bfloat16).requires_grad_() for i in (1, 2))
    weights = torch.ones((5, 2), device=DEV, requires_grad=True)
    out = _path(m, x, ids, w1, w2, weights)
    assert (out == 0).all()
    for g in torch.autograd.grad(out, (x, w1, w2, weights), torch.ones_like(out)):
        assert (g == 0).all()


def test_path_backward_in_a_graph(m):
    """Forward and backward captured together and replayed on other tokens and routes, against eager runs."""
    T, k = 24, 3
    ids, x, weights, dout = (t.to(DEV) for t in _inputs(T, k, 1, True))
    x, dout, weights = x.to(torch.bfloat16), dout.to(torch.bfloat16), weights.float()
    w1, w2 = (_weights(i).to(DEV, torch.bfloat16) for i in (1, 2))

    def step():
        leaves = [t.detach().requires_grad_() for t in (x, w1, w2, weights)]      # new leaves: none lives on outside a step
        out = _path(m, leaves[0], ids, *leaves[1:])
        return [out.detach(), *torch.autograd.grad(out, leaves, dout)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (2, 3, 4):
        for t, v in zip((ids, x, weights, dout), _inputs(T, k, seed, seed != 3)):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        again = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(again, step()))


def test_example_trains_in_fp8(m):
    from fp8_block_scaled_grouped_amd.examples.ragged_experts import RaggedExperts, train
    shape = dict(H=128, I=64, E=8, n_group=4, topk_group=2, topk=2, device=DEV)
    layer, teacher = RaggedExperts(**shape, seed=1, fp8=True), RaggedExperts(**shape, seed=2)
    g = torch.Generator().manual_seed(1)
    x, logits = torch.randn((256, 128), generator=g).to(DEV, torch.bfloat16), torch.randn((256, 8), generator=g).to(DEV)
    assert bool(torch.isfinite(train(layer, teacher, x, logits, 3)).all())
    assert all(p.grad is not None and bool(torch.isfinite(p.grad).all()) and bool(p.grad.abs().sum() > 0) for p in layer.parameters())
    assert layer.pack()(x, logits).shape == x.shape
