"""Token grouping, dispatch and combine on the GPU against the oracle.

Grouping and dispatch move whole numbers and whole values: exact.  moe_combine sums k products in fp32 in a fixed order, each
product and each sum off by at most 2^-24 of the largest magnitude on the way: (k + 2) 2^-24 of the sum of the magnitudes covers
them; a dot product of H terms (H + 2) 2^-24 likewise.  Outputs are rounded once to nearest, and rounding is monotone: an
output lies between the rounded ends of the interval around the oracle's value.
"""
import numpy as np
import pytest
import torch

from oracle import dispatch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def m():
    import fp8_block_scaled_grouped_amd as mod
    mod.lib()
    return mod


def _f64(t):
    return t.detach().cpu().double().numpy()


def _within(got, ref, d, dtype, what):
    lo, hi = (_f64(torch.tensor(v).to(dtype)) for v in (ref - d, ref + d))
    g = _f64(got)
    assert g.shape == ref.shape
    bad = ~((g >= lo) & (g <= hi))
    assert not bad.any(), "%s: %d of %d outside, first at %s: %r not in [%r, %r]" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], lo[bad][0], hi[bad][0])


def _ids(T, k, E, seed, outside=True):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-1 if outside else 0, E + (2 if outside else 0), (T, k), generator=g, dtype=torch.int32)


def _place(T, k, E, seed, outside=True):
    off, rop, por = dispatch.group(_ids(T, k, E, seed, outside).numpy(), E)
    return rop, torch.tensor(rop, dtype=torch.int32, device=DEV), int(off[-1])


def _randn(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


# ------------------------------------------------------------------ grouping
# one workgroup up to 4096 pairs, chunks of 4096 beyond; experts off and on powers of two, up to as many as a workgroup has threads
@pytest.mark.parametrize("T,k,E", [(0, 2, 5), (1, 1, 1), (1, 8, 256), (3, 5, 7), (64, 8, 256), (100, 3, 1024), (512, 8, 64), (4096, 1, 2),
                                   (4097, 1, 3), (700, 6, 257), (3001, 8, 1024), (9000, 7, 33), (40000, 8, 256)])
def test_group(m, T, k, E):
    print("group", T, k, E, flush=True)
    ids = _ids(T, k, E, T + E)
    if T * k > 100000:      # the oracle's loop is long: torch's stable sort
        flat = ids.reshape(-1).long()
        key, order = torch.sort(torch.where((flat >= 0) & (flat < E), flat, E), stable=True)
        n = int((key < E).sum())
        off = torch.searchsorted(key, torch.arange(E + 1)).numpy()
        por = torch.where(key < E, order, -1).numpy()
        rop = np.full(T * k, -1)
        rop[por[:n]] = np.arange(n)
        rop = rop.reshape(T, k)
    else:
        off, rop, por = dispatch.group(ids.numpy(), E)
    wide = torch.full((T, k + 3), 77, dtype=torch.int32)      # rows with a stride
    wide[:, :k] = ids
    for x in (ids.to(DEV), wide.to(DEV)[:, :k]):
        o, r, p = m.moe_group(x, E)
        assert (o.cpu().numpy() == off).all() and (r.cpu().numpy() == rop).all() and (p.cpu().numpy() == por).all()


@pytest.mark.parametrize("T,k,E", [(500, 8, 16), (2000, 8, 16)])
def test_group_of_one_expert_and_of_none(m, T, k, E):
    one = torch.full((T, k), E - 1, dtype=torch.int32, device=DEV)
    o, r, p = m.moe_group(one, E)
    assert o.tolist() == [0] * E + [T * k] and torch.equal(r.flatten(), torch.arange(T * k, device=DEV, dtype=torch.int32))
    assert torch.equal(p, r.flatten())
    o, r, p = m.moe_group(torch.full_like(one, -5), E)
    assert o.tolist() == [0] * (E + 1) and (r == -1).all() and (p == -1).all()


def test_group_into_given_buffers_leaves_the_workspace_reusable(m):
    T, k, E = 3000, 4, 50
    n = m.moe_group_workspace(T, k, E)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)
    out = (torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty((T, k), dtype=torch.int32, device=DEV),
           torch.empty(T * k, dtype=torch.int32, device=DEV))
    for seed in (1, 2):
        ids = _ids(T, k, E, seed)
        got = m.moe_group(ids.to(DEV), E, out, ws)
        ref = dispatch.group(ids.numpy(), E)
        assert all((a.cpu().numpy() == b).all() for a, b in zip(got, ref))
    with pytest.raises(m.Moe355Error):
        m.moe_group(ids.to(DEV), E, out, ws[:n - 4])


# ------------------------------------------------------------------ rows
SHAPES = [(1, 1, 1, 1), (5, 3, 4, 8), (64, 8, 16, 7168 // 8), (33, 2, 5, 7), (16, 4, 16, 256), (40, 6, 9, 1160), (7, 12, 64, 513), (3, 40, 4, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32", "u8"])
@pytest.mark.parametrize("T,k,E,H", SHAPES)
def test_dispatch(m, T, k, E, H, dtype):
    print("dispatch", T, k, E, H, dtype, flush=True)
    rop, drop, n = _place(T, k, E, T * k)
    if dtype == "u8":
        x, kept = torch.randint(0, 256, (T, H), dtype=torch.uint8), torch.randint(0, 256, (T * k, H), dtype=torch.uint8)
    else:
        x, kept = _randn((T, H), dtype, 1), _randn((T * k, H), dtype, 2)
    ref = dispatch.dispatch(x.double().numpy(), rop, kept.double().numpy())
    rows = m.moe_dispatch(x.to(DEV), drop, kept.to(DEV))
    assert (_f64(rows) == ref).all()
    assert (_f64(m.moe_dispatch(x.to(DEV), drop))[:n] == ref[:n]).all()
    # strided tokens and rows, and rows that start off 16 bytes
    big, out = torch.zeros((T, H + 5), dtype=x.dtype, device=DEV), torch.zeros((T * k, H + 3), dtype=x.dtype, device=DEV)
    big[:, 1:H + 1] = x.to(DEV)
    out[:, 2:H + 2] = kept.to(DEV)
    m.moe_dispatch(big[:, 1:H + 1], drop, out[:, 2:H + 2])
    assert (_f64(out[:, 2:H + 2]) == ref).all() and (out[:, :2] == 0).all() and (out[:, H + 2:] == 0).all()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,k,E,H", SHAPES)
def test_combine(m, T, k, E, H, dtype, weighted):
    print("combine", T, k, E, H, dtype, weighted, flush=True)
    rop, drop, n = _place(T, k, E, T * k + 1)
    rows = _randn((T * k, H), dtype, 3)
    rows[n:] = float("nan")        # rows behind the last are not read
    wide = torch.rand((T, k + 2), generator=torch.Generator().manual_seed(4))
    wide[:, :k][torch.tensor(rop) < 0] = float("nan")        # nor the weights of pairs without a row
    w = wide[:, :k]
    ref, mag = dispatch.combine(rows.double().numpy(), rop, w.double().numpy() if weighted else None)
    got = m.moe_combine(rows.to(DEV), drop, wide.to(DEV)[:, :k] if weighted else None)
    _within(got, ref, (k + 2) * 2.0 ** -24 * mag, DT[dtype], "combine")
    big, out = torch.zeros((T * k, H + 1), dtype=rows.dtype, device=DEV), torch.zeros((T, H + 9), dtype=rows.dtype, device=DEV)
    big[:, 1:] = rows.to(DEV)
    m.moe_combine(big[:, 1:], drop, w.to(DEV) if weighted else None, out[:, 1:H + 1])
    assert torch.equal(out[:, 1:H + 1], got) and (out[:, 0] == 0).all() and (out[:, H + 1:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,k,E,H", SHAPES)
def test_combine_grad(m, T, k, E, H, dtype):
    print("combine_grad", T, k, E, H, dtype, flush=True)
    rop, drop, n = _place(T, k, E, T * k + 2)
    rows, dout, kept = _randn((T * k, H), dtype, 5), _randn((T, H), dtype, 6), _randn((T * k, H), dtype, 7)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(8))
    ref, dw, mag = dispatch.combine_grad(dout.double().numpy(), rows.double().numpy(), rop, w.double().numpy(), kept.double().numpy())
    args = dout.to(DEV), rows.to(DEV), drop, w.to(DEV)
    drows, dweights = m.moe_combine_grad(*args, kept.to(DEV))
    _within(drows, ref, 2.0 ** -24 * np.abs(ref), DT[dtype], "drows")
    _within(dweights, dw, (H + 2) * 2.0 ** -24 * mag, torch.float32, "dweights")
    assert (dweights.cpu().numpy()[rop < 0] == 0).all()
    a, none = m.moe_combine_grad(*args, kept.to(DEV), want=(True, False))
    assert none is None and torch.equal(a, drows)
    none, b = m.moe_combine_grad(*args, want=(False, True))
    assert none is None and torch.equal(b, dweights)
    # rows off 16 bytes take element-wise loads: the products are the same, the order of the dot products is not
    big, d2 = torch.zeros((T * k, H + 1), dtype=rows.dtype, device=DEV), torch.zeros((T * k, H + 1), dtype=rows.dtype, device=DEV)
    big[:, 1:] = rows.to(DEV)
    d2[:, 1:] = kept.to(DEV)
    _, b = m.moe_combine_grad(dout.to(DEV), big[:, 1:], drop, w.to(DEV), d2[:, 1:])
    assert torch.equal(d2[:, 1:], drows) and (d2[:, 0] == 0).all()
    _within(b, dw, (H + 2) * 2.0 ** -24 * mag, torch.float32, "dweights off 16 bytes")


def test_places_outside_the_rows_are_left_out(m):
    T, k, H = 6, 3, 40
    rop = torch.tensor([[0, 5, 99], [-1, -7, 4], [3, 2, 1], [6, 2 ** 31 - 1, -2 ** 31], [7, 8, 9], [10, 11, 12]], dtype=torch.int32)
    R = 10
    x, rows, kept = _randn((T, H), "bf16", 1), _randn((R, H), "bf16", 2), _randn((R, H), "bf16", 3)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(4))
    ref = dispatch.dispatch(x.double().numpy(), rop.numpy(), kept.double().numpy())
    assert (_f64(m.moe_dispatch(x.to(DEV), rop.to(DEV), kept.to(DEV))) == ref).all()
    out, mag = dispatch.combine(rows.double().numpy(), rop.numpy(), w.double().numpy())
    _within(m.moe_combine(rows.to(DEV), rop.to(DEV), w.to(DEV)), out, (k + 2) * 2.0 ** -24 * mag, torch.bfloat16, "combine")
    d, dw, mag = dispatch.combine_grad(x.double().numpy(), rows.double().numpy(), rop.numpy(), w.double().numpy(), kept.double().numpy())
    gd, gw = m.moe_combine_grad(x.to(DEV), rows.to(DEV), rop.to(DEV), w.to(DEV), kept.to(DEV))
    _within(gd, d, 2.0 ** -24 * np.abs(d), torch.bfloat16, "drows")
    _within(gw, dw, (H + 2) * 2.0 ** -24 * mag, torch.float32, "dweights")


def test_infinities_and_nan_stay_with_their_token(m):
    T, k, E, H = 12, 3, 4, 64
    rop, drop, _ = _place(T, k, E, 9, outside=False)
    rows = _randn((T * k, H), "bf16", 1)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(2))
    clean = m.moe_combine(rows.to(DEV), drop, w.to(DEV))
    rows[rop[4, 1], 3], rows[rop[7, 0], 5] = float("inf"), float("nan")
    got = m.moe_combine(rows.to(DEV), drop, w.to(DEV))
    assert got[4, 3] == float("inf") and got[7, 5].isnan()
    got[4, 3], got[7, 5] = clean[4, 3], clean[7, 5]
    assert torch.equal(got, clean)


def test_gradients_through_autograd(m):
    T, k, E, H = 20, 3, 6, 48
    _, drop, _ = _place(T, k, E, 5, outside=False)
    x = _randn((T, H), "fp32", 1).to(DEV).requires_grad_()
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(2)).to(DEV).requires_grad_()
    g = _randn((T, H), "fp32", 3).to(DEV)

    def plain(x, w):
        return (w[..., None] * (2.0 * x[:, None, :].expand(-1, k, -1))).sum(1)

    out = m.moe_combine(2.0 * m.moe_dispatch(x, drop), drop, w)
    dx, dw = torch.autograd.grad(out, (x, w), g)
    # the same through torch's own gradients in 64 bits: 2k products and sums, 2H in the dot products
    xd, wd = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    ref = plain(xd, wd)
    rx, rw = torch.autograd.grad(ref, (xd, wd), g.double())
    mag = (2 * w.abs().sum(1, keepdim=True) * g.abs()).detach()
    assert ((dx - rx).abs() <= 2 * (k + 3) * 2.0 ** -24 * mag).all()
    assert ((dw - rw).abs() <= (H + 4) * 2.0 ** -24 * (2 * x.abs() * g.abs()).sum(1, keepdim=True)).all()
    assert ((out - ref).abs() <= (k + 4) * 2.0 ** -24 * plain(x.abs(), w)).all()
    # only what is asked for
    y = m.moe_combine(m.moe_dispatch(x.detach(), drop), drop, w)
    assert torch.autograd.grad(y, w, g)[0].shape == w.shape
    with torch.no_grad():
        assert not m.moe_dispatch(x, drop).requires_grad


@pytest.mark.parametrize("weighted", [False, True])
def test_gradient_of_rows_that_no_pair_has_is_zero(m, weighted):
    rows = _randn((6, 32), "fp32", 1).to(DEV).requires_grad_()
    rop = torch.tensor([[4, -1], [1, 9]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[2.0, 3.0], [4.0, 5.0]], device=DEV) if weighted else None
    g = _randn((2, 32), "fp32", 2).to(DEV)
    torch.full((6, 32), float("nan"), device=DEV)                        # what a new buffer may hold
    (d,) = torch.autograd.grad(m.moe_combine(rows, rop, w), rows, g)
    ref = torch.zeros_like(rows)
    ref[4], ref[1] = g[0] * (2 if weighted else 1), g[1] * (4 if weighted else 1)
    assert torch.equal(d, ref)


def test_rows_past_two_to_the_31_bytes(m):
    """Row offsets are 64 bits: the last rows of a buffer of 4.3 GB, in it and back."""
    T, k, H = 4, 2, 1 << 15
    R = (1 << 32) // (2 * H) + 64
    rows = torch.zeros((R, H), dtype=torch.bfloat16, device=DEV)
    rop = torch.tensor([[R - 1, 0], [R - 2, 1], [R // 2, R // 2 + 1], [R - 64, 7]], dtype=torch.int32, device=DEV)
    x = _randn((T, H), "bf16", 1).to(DEV)
    m.moe_dispatch(x, rop, rows)
    assert torch.equal(rows[rop.long()], x[:, None].expand(-1, k, -1))
    assert torch.equal(m.moe_combine(rows, rop), x * 2)
    w = torch.full((T, k), 0.5, device=DEV)
    d, dw = m.moe_combine_grad(x, rows, rop, w, rows)
    assert torch.equal(rows[rop.long()], (x * 0.5)[:, None].expand(-1, k, -1))


def test_another_stream_and_graph_replays(m):
    T, k, E, H = 300, 4, 16, 256
    s = torch.cuda.Stream()
    ids, x = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    w = torch.empty((T, k), device=DEV)

    def layer():
        off, rop, por = m.moe_group(ids, E)
        rows = m.moe_dispatch(x, rop)
        out = m.moe_combine(rows, rop, w)
        drows, dw = m.moe_combine_grad(x, rows, rop, w, torch.zeros_like(rows))
        return off, rop, por, out, drows, dw

    def fill(seed):
        ids.copy_(_ids(T, k, E, seed))
        x.copy_(_randn((T, H), "bf16", seed))
        w.copy_(torch.rand((T, k), generator=torch.Generator().manual_seed(seed)))

    fill(0)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer()
    for seed in (1, 2, 3):
        fill(seed)
        g.replay()
        torch.cuda.synchronize()
        again = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(again, layer()))


def test_refusals(m):
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    off, rop, por = m.moe_group(ids, 3)
    x = torch.zeros((4, 8), dtype=torch.bfloat16, device=DEV)
    rows, w = m.moe_dispatch(x, rop), torch.ones((4, 2), device=DEV)
    for bad in (lambda: m.moe_group(ids.long(), 3), lambda: m.moe_group(ids.cpu(), 3), lambda: m.moe_group(ids.t(), 3),
                lambda: m.moe_dispatch(x.cpu(), rop), lambda: m.moe_dispatch(x.double(), rop), lambda: m.moe_dispatch(x[:3], rop),
                lambda: m.moe_dispatch(x, rop.long()), lambda: m.moe_dispatch(x, rop.flatten()),
                lambda: m.moe_dispatch(x, rop, rows[:, :4]), lambda: m.moe_dispatch(x, rop, rows.float()),
                lambda: m.moe_combine(rows, rop, w.half()), lambda: m.moe_combine(rows, rop, w[:3]),
                lambda: m.moe_combine(rows.to(torch.uint8), rop), lambda: m.moe_combine(rows, rop, w, x.float()),
                lambda: m.moe_combine_grad(x.float(), rows, rop, w), lambda: m.moe_combine_grad(x[:, :4], rows, rop, w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.Moe355Error):
        m.moe_group(ids, 2000)
