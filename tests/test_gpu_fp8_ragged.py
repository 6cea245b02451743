"""FP8 operands and ragged expert products on the GPU against the 64-bit oracle.

Tolerances.  Codes and scales: exact.  Products: an fp32 sum of n terms in any order is within d = (n + 8) 2^-23 of the sum of
their magnitudes (2^-23 rather than 2^-24 a step, in case the matrix unit truncates; an fp32 scale costs three more
roundings a block, inside the 8 and the factor of two).  The terms are not quite the products: the unit takes them eight at a
time and cuts each to 13 bits below the exponent of the largest (test_unit_cuts_products_of_eight pins that), so each of the other
seven loses less than 2^-13 of the largest, and an eight less than 7 * 2^-13 of (largest |a|) (largest |b|): unit_bound is the
sum of these.  All outputs are held to d + unit_bound; a sample of them to d alone, around the sum of the products as the
unit cuts them (unit_sum).  The output is rounded once to nearest, and rounding is monotone: it lies between the rounded
ends of the interval.
"""
import numpy as np
import pytest
import torch

from oracle import fp8_ragged as o, ragged

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


def _close(got, ref, mag, n, dtype, what="", unit=0.0):
    d = (n + 8) * 2.0 ** -23 * mag + unit
    lo, hi = (_f64(torch.tensor(v).to(DT[dtype])) for v in (ref - d, ref + d))
    g = _f64(got)
    assert g.shape == ref.shape
    bad = ~((g >= lo) & (g <= hi))
    assert not bad.any(), "%s: %d of %d outside, first at %s: %r not in [%r, %r]" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], lo[bad][0], hi[bad][0])


def _randn(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


def _offsets(counts, lead=0):
    return [lead] + (lead + np.cumsum(counts)).tolist()


def _dev(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def _wide_range(shape, dtype, seed):
    """Columns and rows of very different magnitudes, zeros, ties and edge values."""
    x = _randn(shape, "fp32", seed)
    span = 30 if dtype == "bf16" else 4
    x = x * torch.logspace(-span, span / 2, shape[1], base=2) * torch.logspace(span / 4, -span / 4, shape[0], base=2)[:, None]
    x = x.to(DT[dtype])
    if shape[0] > 2 and shape[1] >= 16:
        x[0] = 0
        x[:, 3] = 0
        x[1, :16] = torch.tensor([448, 1, 1.0625, 1.1875, 0.0009765625, 0.0029296875, -0.0, 0, 17, 19, 21, 23, -464, 2 ** -9, 2 ** -10, 3 * 2 ** -10]).to(x.dtype)
        x[2, :8] = torch.finfo(x.dtype).tiny
        x[2, 4:8] = torch.tensor(torch.finfo(x.dtype).smallest_normal).to(x.dtype) / 2
    return x


# ------------------------------------------------------------------ operands
SEGMENTS = [([5], 0, 0), ([0, 128, 0, 1, 127], 0, 0), ([129, 0, 300, 2], 3, 5), ([1] * 40, 130, 7), ([], 4, 0), ([0, 0], 6, 0), ([256, 255, 257], 0, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K", [8, 120, 128, 136, 400])
@pytest.mark.parametrize("counts,lead,tail", SEGMENTS)
def test_quant_ragged(m, counts, lead, tail, K, dtype):
    print("quant_ragged", counts, lead, tail, K, dtype, flush=True)
    off = _offsets(counts, lead)
    R = off[-1] + tail
    x = _wide_range((R, K), dtype, R + K)
    keep = x.clone()
    keep[:off[0]], keep[off[-1]:] = float("nan"), float("nan")       # rows in no segment are not read
    q, s, qt, ts = m.fp8_quant_ragged(keep.to(DEV), _dev(off))
    rq, rs = o.quant_blocks(_f64(x), 1)
    rqt, rts, used = o.quant_columns(_f64(x), off)
    a, b = off[0], off[-1]
    assert (q.cpu().numpy()[a:b] == rq[a:b]).all() and (s.cpu().numpy()[a:b] == rs[a:b]).all()
    assert (qt.cpu().numpy()[used] == rqt[used]).all() and (ts.cpu().numpy()[used] == rts[used]).all()
    q1, s1, none, _ = m.fp8_quant_ragged(keep.to(DEV), _dev(off), columns=False)
    assert none is None and torch.equal(q1[a:b], q[a:b]) and torch.equal(s1[a:b], s[a:b])
    none, _, qt1, ts1 = m.fp8_quant_ragged(keep.to(DEV), _dev(off), rows=False)
    assert none is None and (qt1.cpu().numpy()[used] == rqt[used]).all() and (ts1.cpu().numpy()[used] == rts[used]).all()
    q2, s2, _, _ = m.fp8_quant_ragged(x.to(DEV))
    assert (q2.cpu().numpy() == rq).all() and (s2.cpu().numpy() == rs).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quant_every_value_under_every_scale(m, dtype):
    """Blocks of 127 values under each largest magnitude 448 * 2^e: every value of the 21 binades below it, so subnormal codes,
    all ties and those that round to zero."""
    bits = torch.arange(0, 0x7f80 if dtype == "bf16" else 0x7c00, dtype=torch.int32).to(torch.int16)
    mags = bits.view(DT[dtype]).double()
    rows = []
    for e in range(-126, 120) if dtype == "bf16" else range(-23, 8):
        top = torch.tensor(448.0 * 2.0 ** e, dtype=torch.float64)
        some = mags[(mags <= top) & (mags >= top * 2.0 ** -21)]
        some = torch.cat([some, -some])
        some = torch.nn.functional.pad(some, (0, -some.numel() % 127)).view(-1, 127)
        rows.append(torch.cat([top.expand(some.shape[0], 1), some], 1))
    x64 = torch.cat(rows)
    x = x64.to(DT[dtype])
    assert torch.equal(x.double(), x64)
    rq, rs = o.quant_blocks(x64.numpy(), 1)
    q, s, _, _ = m.fp8_quant_ragged(x.to(DEV), columns=False)
    assert (s.cpu().numpy() == rs).all() and (q.cpu().numpy() == rq).all()
    xt = x.t()[:, :x.shape[0] // 8 * 8].contiguous()                   # the same blocks as columns of 128 rows
    _, _, qt, ts = m.fp8_quant_ragged(xt.to(DEV), _dev([0, 128]), rows=False)
    n = xt.shape[1]
    assert (ts[0].cpu().numpy() == rs[:n, 0]).all() and (qt[0].cpu().numpy() == rq[:n]).all()
    wq, ws = m.fp8_quant_128x128(x[:128].to(DEV)[None])
    rwq, rws = o.quant_blocks(x64.numpy()[:128], 128)
    assert (wq[0].cpu().numpy() == rwq).all() and (ws[0].cpu().numpy() == rws).all()


def test_quant_ragged_strided_rows(m):
    x = _randn((150, 400), "bf16", 1).to(DEV)
    off = _dev([0, 20, 150])
    q, s, qt, ts = m.fp8_quant_ragged(x[:, 64:320], off)
    for a, b in zip((q, s), m.fp8_quant_ragged(x[:, 64:320].contiguous(), off)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_quant_ragged_non_finite_blocks(m, bad):
    off = [0, 100, 260]
    x = _randn((260, 256), "bf16", 2)
    x[100, 130] = bad                    # the first row of the second segment
    q, s, qt, ts = m.fp8_quant_ragged(x.to(DEV), _dev(off))
    rs, (rqt, rts, used) = o.quant_blocks(_f64(x), 1)[1], o.quant_columns(_f64(x), off)
    assert rs[100, 1] == 255 and (rs == 255).sum() == 1 and (rts[used] == 255).sum() == 1
    assert (s.cpu().numpy() == rs).all() and (ts.cpu().numpy()[used] == rts[used]).all()
    ok = np.ones(x.shape, bool)
    ok[100, 128:] = False
    assert (q.cpu().numpy()[ok] == o.quant_blocks(_f64(x), 1)[0][ok]).all()


@pytest.mark.parametrize("fmt", ["e8m0", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("E,N,K", [(1, 16, 8), (3, 128, 128), (2, 144, 264), (1, 304, 128), (2, 16, 400)])
def test_quant_128x128(m, E, N, K, dtype, fmt):
    print("quant_128x128", E, N, K, dtype, fmt, flush=True)
    w = torch.stack([_wide_range((N, K), dtype, N + K + e) for e in range(E)])
    w[0, :, K // 2:] = 0
    q, s, qt, ts = m.fp8_quant_128x128(w.to(DEV), fmt, transposed=True)
    for e in range(E):
        rq, rs = o.quant_blocks(_f64(w[e]), 128, fmt)
        assert (s[e].cpu().numpy() == rs).all() and (q[e].cpu().numpy() == rq).all()
    assert torch.equal(qt, q.transpose(1, 2)) and torch.equal(ts, s.transpose(1, 2))
    q2, s2 = m.fp8_quant_128x128(w.to(DEV), fmt)
    assert torch.equal(q2, q) and torch.equal(s2, s)


@pytest.mark.parametrize("fmt", ["e8m0", "fp32"])
def test_quant_128x128_non_finite_block(m, fmt):
    w = _randn((1, 256, 256), "bf16", 3)
    w[0, 200, 10] = float("nan")
    q, s = m.fp8_quant_128x128(w.to(DEV), fmt)
    rq, rs = o.quant_blocks(_f64(w[0]), 128, fmt)
    assert np.array_equal(s[0].cpu().numpy(), rs, equal_nan=fmt == "fp32") and (rs[1, 0] == 255 if fmt == "e8m0" else np.isnan(rs[1, 0]))
    ok = np.ones((256, 256), bool)
    ok[128:, :128] = False
    assert (q[0].cpu().numpy()[ok] == rq[ok]).all()


# ------------------------------------------------------------------ products
def _pick(n, most=40):
    """Indices spread over n rows, the first and the last among them."""
    return np.unique(np.linspace(0, n - 1, min(n, most)).astype(int)) if n else np.zeros(0, int)


class _Operands:
    """Codes and scales of a product over ragged rows, and their values."""

    def __init__(self, off, xq, xs, wq, ws):
        self.off, self.xq, self.xs, self.wq, self.ws = off, xq, xs, wq, ws
        self.R, self.E, (self.N, self.K) = len(xq), len(wq), wq.shape[1:]
        self.dev = [torch.tensor(t, device=DEV) for t in (xq, xs, wq, ws)]
        self.x, self.w = o.values(xq, xs, 1), o.values(wq, ws, 128)

    def check(self, y, dtype, what):
        """Rows of y in segments against the oracle, all with the unit's bound and a sample without."""
        off = self.off
        ref, mag = ragged.forward(self.x, self.w, off)
        ex = o.each(self.xs, 1, self.R, self.K)
        y = y.detach().cpu()
        for e, (a, b) in enumerate(zip(off, off[1:])):
            if a == b:
                continue
            ew = o.each(self.ws[e], 128, self.N, self.K)
            unit = o.unit_bound(self.xq[a:b], ex[a:b], self.wq[e], ew)
            _close(y[a:b], ref[a:b], mag[a:b], self.K, dtype, "%s of expert %d" % (what, e), unit)
            r, c = a + _pick(b - a), _pick(self.N)
            cut = o.unit_sum(self.xq[r], ex[r], self.wq[e][c], ew[c])
            _close(y[r][:, c], cut, mag[r][:, c], self.K, dtype, "sample of %s of expert %d" % (what, e))


def _operands(counts, E, N, K, fmt, seed, lead=0, tail=0):
    off = _offsets(counts, lead)
    R = off[-1] + tail
    x, w = _wide_range((R, K), "fp16", seed).double(), _randn((E, N, K), "bf16", seed + 1, 0.1).double()
    packed = [o.quant_blocks(e.numpy(), 128, fmt) for e in w]
    return _Operands(off, *o.quant_blocks(x.numpy(), 1, fmt), np.stack([p[0] for p in packed]), np.stack([p[1] for p in packed]))


def _check_wgrad(dw, dyt, dys, xt, xs, off, most, dtype):
    ref, mag = o.wgrad(dyt, dys, xt, xs, off)
    dw = dw.detach().cpu()
    for e in range(len(off) - 1):
        dq, ds = o.column_codes(dyt, dys, off, e)
        q, s = o.column_codes(xt, xs, off, e)
        _close(dw[e], ref[e], mag[e], most, dtype, "dw of expert %d" % e, o.unit_bound(dq, ds, q, s))
        r, c = _pick(len(dq)), _pick(len(q))
        _close(dw[e][r][:, c], o.unit_sum(dq[r], ds[r], q[c], s[c]), mag[e][r][:, c], most, dtype, "sample of dw of expert %d" % e)


# (rows of the experts, E, N, K): every tile (64, 128 and 256 wide), odd rows, columns and blocks, one block and many
FWD = [([1], 1, 8, 16), ([3, 0, 17, 64], 4, 136, 272), ([65, 1, 0, 70], 4, 72, 128), ([200, 100, 0, 211], 4, 2568, 144),
       ([400, 130, 129, 300], 4, 2600, 400), ([1300, 1260], 2, 5128, 144), ([700, 0, 900, 500], 4, 4104, 272)]


@pytest.mark.parametrize("fmt", ["e8m0", "fp32"])
@pytest.mark.parametrize("counts,E,N,K", FWD)
def test_product(m, counts, E, N, K, fmt):
    print("grouped_gemm_fp8", counts, E, N, K, fmt, flush=True)
    ops = _operands(counts, E, N, K, fmt, N + K, lead=2, tail=3)
    off, (xq, xs, wq, ws) = ops.off, ops.dev
    a, b = off[0], off[-1]
    for i, dtype in enumerate(("bf16", "fp16")):
        y = torch.full((ops.R, N), 7.0, dtype=DT[dtype], device=DEV)
        lay = ({}, {"scale_layout": "kblock"})[i]
        got = m.grouped_gemm_fp8(xq, xs.t().contiguous() if i else xs, wq, ws, _dev(off), y, **lay)
        assert got is y and (y[:a] == 7).all() and (y[b:] == 7).all()
        ops.check(y, dtype, "y")
    # strided rows in and out
    big, out = torch.zeros((ops.R, K + 48), dtype=torch.uint8, device=DEV), torch.zeros((ops.R, N + 16), dtype=torch.bfloat16, device=DEV)
    big[:, 16:16 + K] = xq
    m.grouped_gemm_fp8(big[:, 16:16 + K], xs, wq, ws, _dev(off), out[:, 8:8 + N])
    assert torch.equal(out[a:b, 8:8 + N], m.grouped_gemm_fp8(xq, xs, wq, ws, _dev(off))[a:b])
    assert (out[:, :8] == 0).all() and (out[:, 8 + N:] == 0).all() and (out[:a] == 0).all() and (out[b:] == 0).all()


@pytest.mark.parametrize("fmt", ["e8m0", "fp32"])
@pytest.mark.parametrize("counts,E,N,K", [([3, 0, 17, 64], 4, 136, 7168), ([400, 130, 129, 300], 4, 2600, 2048), ([1300, 1260], 2, 5128, 1168)])
def test_product_of_whole_numbers_is_exact(m, counts, E, N, K, fmt):
    """Whole numbers up to 4 under scales of one: the sums stay below 16 * 7168 < 2^24, exact in fp32 in any order, so every bit of
    the output is known (a matrix unit that dropped low bits would show)."""
    off, R, g = _offsets(counts), sum(counts), np.random.default_rng(K)
    x, w = g.integers(-4, 5, (R, K)), g.integers(-4, 5, (E, N, K))
    one = lambda *shape: torch.full(shape, 127 if fmt == "e8m0" else 1, dtype=torch.uint8 if fmt == "e8m0" else torch.float32, device=DEV)
    codes = lambda t: torch.tensor(o.fp8.encode(t.astype(np.float32)), device=DEV)
    y = m.grouped_gemm_fp8(codes(x), one(R, -(-K // 128)), codes(w), one(E, -(-N // 128), -(-K // 128)), _dev(off))
    ref = np.concatenate([x[a:b].astype(np.float32) @ w[e].T.astype(np.float32) for e, (a, b) in enumerate(zip(off, off[1:]))])
    assert torch.equal(y.cpu(), torch.tensor(ref).to(torch.bfloat16))


WGRAD = [([1], 1, 8, 8), ([5, 0, 130, 64], 4, 40, 264), ([128, 256, 0, 127], 4, 264, 136), (([7, 0, 140] * 8), 24, 264, 264),
         (([3, 150, 0, 20] * 32), 128, 264, 264)]


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("counts,E,N,K", WGRAD)
def test_wgrad(m, counts, E, N, K, out):
    print("grouped_gemm_fp8_wgrad", len(counts), E, N, K, out, flush=True)
    off = _offsets(counts, 5)
    R = off[-1] + 9
    dy, x = _wide_range((R, N), "fp16", 1), _randn((R, K), "fp16", 2)
    dyt, dys, used = o.quant_columns(_f64(dy), off)
    xt, xs, _ = o.quant_columns(_f64(x), off)
    for t, fill in ((dyt, 0x7f), (xt, 0x7f), (dys, 255), (xs, 255)):       # blocks that no expert has are not read
        t[~used] = fill
    args = [torch.tensor(t, device=DEV) for t in (dyt, dys, xt, xs)]
    dw = torch.full((E, N, K), float("nan"), dtype=DT[out], device=DEV)
    got = m.grouped_gemm_fp8_wgrad(*args, _dev(off), R, dw)
    assert got is dw
    _check_wgrad(dw, dyt, dys, xt, xs, off, max(counts), out)
    assert (dw[[i for i, c in enumerate(counts) if c == 0]] == 0).all()


def test_wgrad_without_rows_is_zero(m):
    z = torch.zeros
    dw = m.grouped_gemm_fp8_wgrad(z((3, 16, 128), dtype=torch.uint8, device=DEV), z((3, 16), dtype=torch.uint8, device=DEV),
                                  z((3, 24, 128), dtype=torch.uint8, device=DEV), z((3, 24), dtype=torch.uint8, device=DEV),
                                  _dev([0, 0, 0, 0]), 0)
    assert dw.shape == (3, 16, 24) and (dw == 0).all()


def test_unit_cuts_products_of_eight(m):
    """What the tolerances rest on: a product of e = 16 next to a small one among the same eight leaves that one's multiples of
    2^(16 - 13), cut towards zero, and takes nothing from the next eight; sums of the eights keep fp32's 24 bits."""
    def dw(a, b):       # rows of 128 values -> their products' sum
        enc = lambda v: torch.stack([torch.tensor(v).to(torch.float8_e4m3fn).view(torch.uint8), torch.zeros(128, dtype=torch.uint8)])
        rep = lambda t: t[:, None].expand(2, 8, 128).contiguous().to(DEV)
        one = torch.full((2, 8), 127, dtype=torch.uint8, device=DEV)
        return m.grouped_gemm_fp8_wgrad(rep(enc(a)), one, rep(enc(b)), one, _dev([0, 128]), 128)[0, 0, 0].item()

    def two(at, u, v, first=(256.0, 256.0)):
        a, b = np.zeros(128), np.zeros(128)
        a[0], b[0] = first
        a[at], b[at] = u, v
        got = dw(a, b)
        enc = lambda t: o.fp8.encode(t.astype(np.float32))[None]
        assert got == np.float32(o.unit_sum(enc(a), np.ones((1, 128)), enc(b), np.ones((1, 128)))[0, 0]), (at, u, v)
        return got - first[0] * first[1]

    assert two(1, 4.0, 7.0) == 24 and two(7, -4.0, 7.0) == -24 and two(3, 2.0, 3.5) == 0 and two(5, 2.0, 4.0) == 8
    assert two(8, 4.0, 7.0) == 28 and two(127, 2.0 ** -3, 2.0 ** -4) == 2.0 ** -7
    assert two(1, 2.0 ** -5, 2.0 ** -6, (2.0 ** -9, 256.0)) == 2.0 ** -11 and two(1, 2.0 ** -6, 2.0 ** -6, (2.0 ** -9, 256.0)) == 0
    assert two(1, 2.0 ** -9, 2.0 ** -9, (0.0, 256.0)) == 2.0 ** -18


@pytest.mark.parametrize("big", [64.0, 256.0])
def test_fp32_sums_keep_every_bit(m, big):
    """One large product and many ones (the seven beside it in its eight, which the unit may cut, left out): the sum is exact in fp32 and
    shows sums that are held in fewer bits."""
    K, N, R = 2048, 64, 40
    x, w = torch.ones((R, K)), torch.ones((1, N, K))
    x[:, :8] = 0
    x[:, 5], w[0, :, 5] = big, big
    enc = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)
    ref = big * big + K - 8
    for one, dt in ((127, torch.uint8), (1.0, torch.float32)):
        y = m.grouped_gemm_fp8(enc(x).to(DEV), torch.full((R, K // 128), one, dtype=dt, device=DEV), enc(w).to(DEV),
                               torch.full((1, 1, K // 128), one, dtype=dt, device=DEV), _dev([0, R]))
        assert (y.float() == torch.tensor(ref).to(torch.bfloat16).float().item()).all()
    # over rows, into fp32: every bit
    d, x = torch.ones((K, 24)), torch.ones((K, 16))
    d[:8] = 0
    d[5], x[5] = big, big
    pack = lambda t: enc(t).view(K // 128, 128, t.shape[1]).transpose(1, 2).contiguous()
    pad = lambda t: torch.cat([t, torch.full((1, *t.shape[1:]), 0x7f, dtype=torch.uint8)]).to(DEV)
    ones = lambda c: torch.full((K // 128 + 1, c), 127, dtype=torch.uint8, device=DEV)
    dw = m.grouped_gemm_fp8_wgrad(pad(pack(d)), ones(24), pad(pack(x)), ones(16), _dev([0, K]), K)
    assert (dw == ref).all(), dw.flatten()[0]


@pytest.mark.parametrize("fmt", ["e8m0", "fp32"])
def test_non_finite_values_stay_in_their_rows(m, fmt):
    counts, E, N, K = [70, 130, 66], 3, 200, 256
    ops = _operands(counts, E, N, K, fmt, 1)
    off, (xq, xs, wq, ws) = ops.off, ops.dev
    clean = m.grouped_gemm_fp8(xq, xs, wq, ws, _dev(off))
    nan = 255 if fmt == "e8m0" else float("nan")
    xs[70, 1] = nan                                  # the first row of expert 1
    got = m.grouped_gemm_fp8(xq, xs, wq, ws, _dev(off))
    assert got[70].isnan().all()
    keep = torch.arange(len(xq), device=DEV) != 70
    assert torch.equal(got[keep], clean[keep])
    ws[2, 1, 0] = nan                                # columns 128.. of expert 2
    got = m.grouped_gemm_fp8(xq, xs, wq, ws, _dev(off))
    assert got[200:, 128:].isnan().all() and torch.equal(got[200:, :128], clean[200:, :128])
    keep[200:] = False
    assert torch.equal(got[keep], clean[keep])


def test_scale_bytes_from_end_to_end(m):
    """Every pair of bytes whose product is an fp32 number, on codes of one."""
    K, N = 128, 8
    one = torch.full((1, K), 0x38, dtype=torch.uint8, device=DEV)
    a = torch.arange(0, 255, dtype=torch.uint8, device=DEV)
    for b in (0, 1, 100, 127, 200, 254):
        y = m.grouped_gemm_fp8(one.expand(255, K).contiguous(), a[:, None], one.expand(1, N, K).contiguous(),
                               torch.full((1, 1, 1), b, dtype=torch.uint8, device=DEV), _dev([0, 255]))
        ex, got = np.arange(255) + (b - 254 + 7), _f64(y[:, 0])
        normal = (ex >= -126) & (ex <= 127)           # below, the matrix unit may flush
        assert (got[normal] == np.ldexp(1.0, ex[normal])).all(), b
        assert not np.isfinite(got[ex > 127]).any()
        assert ((got[ex < -126] == 0) | (got[ex < -126] == np.ldexp(1.0, ex[ex < -126]))).all()


def test_malformed_offsets_write_only_inside(m):
    """Offsets that are negative, too large or decrease are cut to [0, R]: no row outside the output is touched."""
    E, N, K, R = 4, 136, 144, 90
    xq, xs, wq, ws = _operands([R], E, N, K, "e8m0", 4).dev
    x = _randn((R, K), "bf16", 1).to(DEV)
    for off in ([-5, 20, 300, 10, 80], [100, 50, 0, -1, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1, 0, 90, 40]):
        base = torch.full((R + 8, N), 3.0, dtype=torch.bfloat16, device=DEV)
        m.grouped_gemm_fp8(xq, xs, wq, ws, _dev(off), base[4:4 + R])
        assert (base[:4] == 3).all() and (base[4 + R:] == 3).all()
        q, s, qt, ts = m.fp8_quant_ragged(x, _dev(off))
        dw = m.grouped_gemm_fp8_wgrad(torch.zeros_like(qt), torch.zeros_like(ts), torch.zeros_like(qt), torch.zeros_like(ts), _dev(off), R)
        torch.cuda.synchronize()
        assert (dw == 0).all()


# ------------------------------------------------------------------ the linear layer
LINEAR = [([40, 0, 3, 129], 4, 48, 32), ([130, 128, 1, 0, 70], 5, 144, 272), ([300, 500], 2, 1040, 528)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,E,N,K", LINEAR)
def test_linear_and_its_gradients(m, counts, E, N, K, dtype):
    print("grouped_linear_fp8", counts, E, N, K, dtype, flush=True)
    off = _offsets(counts)
    R = off[-1]
    x, w, dy = _randn((R, K), dtype, 1), _randn((E, N, K), dtype, 2, 0.05), _randn((R, N), dtype, 3, 0.01)
    xd, wd = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    y = m.grouped_linear_fp8(xd, wd, _dev(off))
    dx, dw = torch.autograd.grad(y, (xd, wd), dy.to(DEV))
    assert y.dtype == dx.dtype == dw.dtype == DT[dtype]
    packed = [o.quant_blocks(_f64(e), 128) for e in w]
    wq, ws = np.stack([p[0] for p in packed]), np.stack([p[1] for p in packed])
    _Operands(off, *o.quant_blocks(_f64(x), 1), wq, ws).check(y, dtype, "y")
    wt, wst = (np.ascontiguousarray(t.swapaxes(1, 2)) for t in (wq, ws))
    _Operands(off, *o.quant_blocks(_f64(dy), 1), wt, wst).check(dx, dtype, "dx")
    _check_wgrad(dw, *o.quant_columns(_f64(dy), off)[:2], *o.quant_columns(_f64(x), off)[:2], off, max(counts), dtype)
    # one gradient alone
    y = m.grouped_linear_fp8(xd, w.to(DEV), _dev(off))
    assert torch.equal(torch.autograd.grad(y, xd, dy.to(DEV))[0], dx)
    y = m.grouped_linear_fp8(x.to(DEV), wd, _dev(off))
    assert torch.equal(torch.autograd.grad(y, wd, dy.to(DEV))[0], dw)
    # a gradient that starts off 16 bytes and one that is broadcast
    odd = torch.zeros(R * N + 1, dtype=DT[dtype], device=DEV)[1:].view(R, N).copy_(dy)
    y = m.grouped_linear_fp8(xd, wd, _dev(off))
    assert torch.equal(torch.autograd.grad(y, xd, odd)[0], dx)
    y = m.grouped_linear_fp8(xd, wd, _dev(off))
    s = torch.autograd.grad(y.sum(), xd)[0]
    y = m.grouped_linear_fp8(xd, wd, _dev(off))
    assert torch.equal(s, torch.autograd.grad(y, xd, torch.ones_like(y))[0])


def test_linear_without_rows_with_strided_rows_and_twice(m):
    E, N, K = 3, 48, 32
    w = _randn((E, N, K), "bf16", 1).to(DEV).requires_grad_()
    x = torch.zeros((0, K), dtype=torch.bfloat16, device=DEV, requires_grad=True)
    y = m.grouped_linear_fp8(x, w, _dev([0, 0, 0, 0]))
    dx, dw = torch.autograd.grad(y, (x, w), torch.zeros_like(y))
    assert y.shape == (0, N) and dx.shape == (0, K) and dw.shape == w.shape and (dw == 0).all()
    # rows with a stride, rows in no segment (their outputs and gradients are anything), and a graph that is run twice
    wide, dy, off = _randn((70, 64), "bf16", 2).to(DEV), _randn((70, N), "bf16", 3).to(DEV), _dev([10, 10, 40, 60])
    a, b = wide[:, 16:48].requires_grad_(), wide[:, 16:48].detach().contiguous().requires_grad_()
    ya, yb = m.grouped_linear_fp8(a, w, off), m.grouped_linear_fp8(b, w, off)
    ga = torch.autograd.grad(ya, (a, w), dy, retain_graph=True)
    twice, gb = torch.autograd.grad(ya, (a, w), dy), torch.autograd.grad(yb, (b, w), dy)
    assert torch.equal(ya[10:60], yb[10:60])
    for g in (twice, gb):
        assert torch.equal(ga[0][10:60], g[0][10:60]) and torch.equal(ga[1], g[1])
    # no experts: no row has a segment
    none = m.grouped_linear_fp8(b.detach(), torch.zeros((0, N, K), dtype=torch.bfloat16, device=DEV), _dev([0]))
    assert none.shape == (70, N)
    for bad in (lambda: m.grouped_linear_fp8(b, w[:, :, :16], off), lambda: m.grouped_linear_fp8(b, w.transpose(1, 2), off),
                lambda: m.grouped_linear_fp8(b, w, off[:2]), lambda: m.grouped_linear_fp8(b, w, off.long()),
                lambda: m.grouped_linear_fp8(b[None], w, off), lambda: m.grouped_linear_fp8(b.float(), w.float(), off),
                lambda: m.grouped_linear_fp8(b, w[:, ::2], off)):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros((2, 40, K), dtype=torch.bfloat16, device=DEV)       # N no multiple of 16: the gradient for x has no codes
    with pytest.raises(m.Moe355Error):
        m.grouped_linear_fp8(b, odd, _dev([0, 10, 70]))


def test_linear_without_gradients_keeps_nothing_for_them(m):
    E, N, K, R = 4, 1024, 2048, 256
    x, w = _randn((R, K), "bf16", 1).to(DEV).requires_grad_(), _randn((E, N, K), "bf16", 2).to(DEV).requires_grad_()
    off, peak, out = _dev([0, 64, 128, 192, R]), [], []
    for grad in (True, False):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        with torch.set_grad_enabled(grad):
            out.append(m.grouped_linear_fp8(x, w, off))
        peak.append(torch.cuda.max_memory_allocated() - before)
    assert out[0].requires_grad and not out[1].requires_grad and torch.equal(*out)
    assert peak[1] <= peak[0] - E * N * K                                # the weights' codes transposed


def test_linear_and_gradients_captured(m):
    """Forward and backward in one graph, on leaves made for each run."""
    E, N, K, R = 4, 144, 272, 300
    x, dy, w = (torch.empty(s, dtype=torch.bfloat16, device=DEV) for s in ((R, K), (R, N), (E, N, K)))
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)

    def step():
        a, b = x.detach().requires_grad_(), w.detach().requires_grad_()
        y = m.grouped_linear_fp8(a, b, off)
        return (y.detach(),) + torch.autograd.grad(y, (a, b), dy)

    def fill(i, counts):
        x.copy_(_randn((R, K), "bf16", i))
        dy.copy_(_randn((R, N), "bf16", i + 9))
        w.copy_(_randn((E, N, K), "bf16", i + 20, 0.05))
        off.copy_(_dev(_offsets(counts)))

    fill(0, [100, 30, 0, 170])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i, counts in ((1, [0, 150, 150, 0]), (2, [300, 0, 0, 0]), (3, [1, 128, 129, 42])):
        fill(i, counts)
        g.replay()
        torch.cuda.synchronize()
        again = [t.clone() for t in got]
        assert all(torch.equal(p, q) for p, q in zip(again, step()))


def test_gradients_against_differences(m):
    """On values that quantisation leaves alone the loss is linear in x and in w, so a difference along any direction
    of such values is the gradient.  All is whole numbers: x + u and w + u up to 4, |y| <= 4 * 2 * 16, |dx| <= 2 * 2 * 32 and
    |dw| <= 2 * 2 * 45, which bf16 holds (up to 256)."""
    counts, E, N, K = [30, 0, 45], 3, 32, 16
    off, g = _dev(_offsets(counts)), torch.Generator().manual_seed(1)
    R = sum(counts)
    r = lambda *shape: torch.randint(-2, 3, shape, generator=g).to(DEV, torch.bfloat16)
    x, w, dy, ux, uw = r(R, K), r(E, N, K), r(R, N), r(R, K), r(E, N, K)
    xd, wd = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(m.grouped_linear_fp8(xd, wd, off), (xd, wd), dy)
    loss = lambda a, b: (m.grouped_linear_fp8(a, b, off).double() * dy.double()).sum().item()
    assert loss(x + ux, w) - loss(x, w) == (dx.double() * ux.double()).sum().item()
    assert loss(x, w + uw) - loss(x, w) == (dw.double() * uw.double()).sum().item()


def test_another_stream_and_graph_replays(m):
    counts = ([100, 30, 0, 170], [0, 150, 150, 0], [300, 0, 0, 0])
    E, N, K, R = 4, 144, 272, 300
    x, dy = torch.empty((R, K), dtype=torch.bfloat16, device=DEV), torch.empty((R, N), dtype=torch.bfloat16, device=DEV)
    w = _randn((E, N, K), "bf16", 1, 0.05).to(DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)

    def step():
        q, s, qt, ts = m.fp8_quant_ragged(x, off)
        p = m.fp8_quant_128x128(w, transposed=True)
        y = m.grouped_gemm_fp8(q, s, p[0], p[1], off)
        dq, ds, dt, dts = m.fp8_quant_ragged(dy, off)
        return y, m.grouped_gemm_fp8(dq, ds, p[2], p[3], off), m.grouped_gemm_fp8_wgrad(dt, dts, qt, ts, off, R)

    def fill(i):
        x.copy_(_randn((R, K), "bf16", i))
        dy.copy_(_randn((R, N), "bf16", i + 9))
        off.copy_(_dev(_offsets(counts[i])))

    fill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(other, step()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in (1, 2, 0):
        fill(i)
        g.replay()
        torch.cuda.synchronize()
        again = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(again, step()))


def test_refusals(m):
    xq, xs, wq, ws = _operands([4, 5], 2, 16, 32, "e8m0", 1).dev
    d = _dev([0, 4, 9])
    x = torch.zeros((9, 32), dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: m.grouped_gemm_fp8(xq.cpu(), xs, wq, ws, d), lambda: m.grouped_gemm_fp8(xq, xs.float(), wq, ws, d),
                lambda: m.grouped_gemm_fp8(xq, xs[:5], wq, ws, d), lambda: m.grouped_gemm_fp8(xq, xs, wq[:, :, :16], ws, d),
                lambda: m.grouped_gemm_fp8(xq, xs, wq, ws, d.long()), lambda: m.grouped_gemm_fp8(xq, xs, wq, ws, d[:2]),
                lambda: m.grouped_gemm_fp8(xq, xs, wq, ws, d, out_dtype=torch.float32),
                lambda: m.grouped_gemm_fp8(xq, xs, wq, ws, d, scale_layout="column"),
                lambda: m.fp8_quant_ragged(x.float(), d), lambda: m.fp8_quant_ragged(x, rows=False),
                lambda: m.fp8_quant_128x128(x), lambda: m.fp8_quant_128x128(x[None], "int8"),
                lambda: m.grouped_linear_fp8(x, torch.zeros((2, 16, 32), dtype=torch.float16, device=DEV), d),
                lambda: m.grouped_gemm_fp8_wgrad(xq, xs, xq, xs, d, 9)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: m.fp8_quant_ragged(x[:, :12], d), lambda: m.fp8_quant_128x128(x[None], transposed=True),
                lambda: m.grouped_gemm_fp8(xq[:, :24], xs, wq[:, :, :24].contiguous(), ws, d)):
        with pytest.raises(m.Moe355Error):
            bad()


def _padded(t, off, most):
    """[R, C] -> [E, most, C] in fp32, zeros behind each expert's rows."""
    r = off[:-1, None] + torch.arange(most, device=DEV)
    return torch.where((r < off[1:, None])[..., None], t.float()[r.clamp(max=max(len(t) - 1, 0))], 0.0)


@pytest.mark.parametrize("E,R,N,K", [(513, 1500, 24, 32), (1500, 700, 136, 144), (65535, 70000, 8, 16), (600, 1200, 4104, 16), (5000, 33000, 520, 16),
                                     (1500, 40000, 264, 272)])
def test_many_experts_and_many_tiles_are_exact(m, E, R, N, K):
    """More experts than a workgroup's table has entries, and more tiles than its stream holds: grids past the CUs.  Whole numbers up to 2
    under scales of one, so every sum is exact: |y| <= 4 * 272 needs no rounding in fp32, and both sides round alike."""
    g = torch.Generator().manual_seed(E)
    c = torch.bincount(torch.randint(0, E, (R,), generator=g), minlength=E)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), c.cumsum(0)]).to(DEV)
    x, w = torch.randint(-2, 3, (R, K), generator=g).to(DEV), torch.randint(-2, 3, (E, N, K), generator=g, dtype=torch.int8).to(DEV)
    table = torch.tensor([0xc0, 0xb8, 0, 0x38, 0x40], dtype=torch.uint8, device=DEV)          # -2 .. 2
    one = lambda *shape: torch.full(shape, 127, dtype=torch.uint8, device=DEV)
    y = m.grouped_gemm_fp8(table[x + 2], one(R, -(-K // 128)), table[w.int() + 2], one(E, -(-N // 128), -(-K // 128)), off.int())
    most = int(c.max())
    ref = torch.bmm(_padded(x, off, most), w.float().transpose(1, 2).contiguous())
    e = torch.repeat_interleave(torch.arange(E, device=DEV), c.to(DEV))
    assert torch.equal(y, ref[e, torch.arange(R, device=DEV) - off[e]].to(torch.bfloat16))


@pytest.mark.parametrize("E,R,N,K", [(513, 1500, 24, 32), (9000, 12000, 136, 136), (65535, 70000, 8, 16)])
def test_gradients_of_many_experts_are_exact(m, E, R, N, K):
    g = torch.Generator().manual_seed(E)
    c = torch.bincount(torch.randint(0, E, (R,), generator=g), minlength=E)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), c.cumsum(0)]).to(DEV)
    x, dy = (torch.randint(-2, 3, (R, n), generator=g).to(DEV) for n in (K, N))
    xt, dyt = (m.fp8_quant_ragged(t.to(torch.bfloat16), off.int(), rows=False)[2:] for t in (x, dy))
    dw = m.grouped_gemm_fp8_wgrad(*dyt, *xt, off.int(), R, out_dtype=torch.bfloat16)
    most = int(c.max())
    assert most * 4 <= 256                                                # bf16 holds every sum
    ref = torch.bmm(_padded(dy, off, most).transpose(1, 2).contiguous(), _padded(x, off, most))
    assert torch.equal(dw.float(), ref)


def test_row_offsets_past_two_to_the_32(m):
    """The last rows of codes, outputs and transposed blocks whose buffers pass 4 GiB."""
    E, N, K = 3, 16, 1 << 15
    R = (1 << 32) // K + 300
    off = [0, R - 260, R - 130, R]
    x8 = torch.zeros((R, K), dtype=torch.uint8, device=DEV)
    x8[R - 260:] = 0x38                                   # ones
    x8[R - 1, ::2] = 0xb8
    xs = torch.full((1, 1), 127, dtype=torch.uint8, device=DEV).expand(R, K // 128)
    w8 = torch.full((E, N, K), 0x38, dtype=torch.uint8, device=DEV)
    ws = torch.full((E, 1, K // 128), 127, dtype=torch.uint8, device=DEV)
    ws[2] = 128
    y = m.grouped_gemm_fp8(x8, xs, w8, ws, _dev(off))
    assert (y[:R - 260] == 0).all() and (y[R - 260:R - 130] == K).all() and (y[R - 130:R - 1] == 2 * K).all() and (y[R - 1] == 0).all()


class _Guarded:
    """A tensor inside a larger allocation whose other bytes must stay."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.base, self.n = torch.full((n + 2048,), 0xA5, dtype=torch.uint8, device=DEV), n
        self.t = self.base[1024:1024 + n].view(dtype).view(shape)

    def intact(self):
        return bool((self.base[:1024] == 0xA5).all()) and bool((self.base[1024 + self.n:] == 0xA5).all())


@pytest.mark.parametrize("counts,N,K", [([1], 8, 16), ([3, 0, 17, 64], 136, 272), ([400, 130, 129, 300], 2600, 400), ([1300, 1260], 5128, 144),
                                        ([30, 41, 0, 38] * 16, 264, 1040), ([7, 0, 140] * 8, 264, 272)])
def test_outputs_stay_inside_their_buffers(m, counts, N, K):
    E, off = len(counts), _offsets(counts)
    R = off[-1]
    g = torch.Generator().manual_seed(N)
    code = lambda *s: torch.randint(0, 0x7f, s, generator=g, dtype=torch.uint8).to(DEV)
    for e8 in (True, False):
        one = lambda *s: torch.full(s, 127 if e8 else 1, dtype=torch.uint8 if e8 else torch.float32, device=DEV)
        y = _Guarded((R, N), torch.bfloat16)
        m.grouped_gemm_fp8(code(R, K), one(R, -(-K // 128)), code(E, N, K), one(E, -(-N // 128), -(-K // 128)), _dev(off), y.t)
        assert y.intact()
    blocks = m.fp8_ragged_blocks(R, E)
    s8 = lambda c: torch.full((blocks, c), 127, dtype=torch.uint8, device=DEV)
    for dt in DT.values():
        dw = _Guarded((E, N, K), dt)
        m.grouped_gemm_fp8_wgrad(code(blocks, N, 128), s8(N), code(blocks, K, 128), s8(K), _dev(off), R, dw.t)
        assert dw.intact()
    x = _randn((R, K), "bf16", 1).to(DEV)
    out = [_Guarded((R, K), torch.uint8), _Guarded((-(-K // 128), R), torch.uint8), _Guarded((blocks, K, 128), torch.uint8),
           _Guarded((blocks, K), torch.uint8)]
    q, s, qt, ts = (o.t.data_ptr() for o in out)
    assert m.lib().fp8_quant_ragged(x.data_ptr(), 0, K, _dev(off).data_ptr(), R, E, K, q, K, s, 1, R, qt, ts,
                                    torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert all(o.intact() for o in out)
