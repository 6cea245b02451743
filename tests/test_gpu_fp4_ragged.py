"""4-bit weights with group scales and ragged expert products on the GPU against the 64-bit oracle.

Tolerances.  Codes, scales and unpacked values: exact.  Products: an fp32 sum of n products in any
order is within d = (n + 8) 2^-23 of the sum of their magnitudes (2^-23 rather than 2^-24 a step, in
case the matrix unit truncates), and the output is rounded once to nearest: rounding is monotone, so
the output lies between the rounded ends of [reference - d, reference + d].
"""
import numpy as np
import pytest
import torch

from oracle import fp4, ragged

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def m():
    import fp8_block_scaled_grouped_amd as mod
    mod.lib()
    return mod


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _close(got, ref, mag, n, dtype, what=""):
    d = (n + 8) * 2.0 ** -23 * mag
    lo, hi = (_f64(torch.tensor(v).to(DT[dtype])) for v in (ref - d, ref + d))
    g = _f64(got)
    assert g.shape == ref.shape
    bad = ~((g >= lo) & (g <= hi))
    assert not bad.any(), "%s: %d of %d outside, first at %s: %r not in [%r, %r]" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], lo[bad][0], hi[bad][0])


def _randn(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


def _offsets(counts):
    return [0] + np.cumsum(counts).tolist()


def _dev_offsets(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ pack and unpack
def _quant_input(rows, K, dtype, seed):
    w = _randn((rows, K), dtype, seed, 0.02)
    lo = 2.0 ** -126 if dtype == "bf16" else 2.0 ** -24
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, -0.25, -0.0, 0.0, -5.0, -6.0, 4.0])
    w[0] = 0
    w[1, :16] = edge.to(w.dtype)                    # with amax 7.5 and, in the next group, amax 6
    if K >= 160:
        w[1, 128:144] = torch.where(edge.abs() > 6, 6.0, edge).to(w.dtype)
    w[2] = (w[2].float() * 0 + lo * 3).to(w.dtype)  # scales at the bottom of the range
    w[2, ::3] = 0
    w[3] *= 3e4 if dtype == "fp16" else 1e37
    w[4, 5], w[4, 40 % K] = float("nan"), float("-inf")
    w[5] = torch.where(torch.arange(K) % 7 == 0, -0.0, 0.0).to(w.dtype)
    return w


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["fp32", "e8m0"])
@pytest.mark.parametrize("group,rows,K", [(32, 37, 96), (64, 9, 160), (128, 300, 416), (128, 6, 32), (32, 64, 7168)])
def test_quant_and_dequant_bit_exact(m, dtype, fmt, group, rows, K):
    print("fp4 quant", dtype, fmt, group, rows, K, flush=True)
    w = _quant_input(rows, K, dtype, rows + K)
    q, s = m.fp4_quant_groups(w.to(DEV), group, fmt)
    rq, rs = fp4.quant_groups(w.float().numpy(), group, fmt == "e8m0")
    gs = s.cpu().numpy()
    assert np.array_equal(gs, rs, equal_nan=fmt == "fp32")
    finite = np.repeat(np.isfinite(fp4.scale_values(rs)), group, -1)[:, :K]
    assert np.array_equal(np.where(finite, fp4.unpack(q.cpu().numpy()), 0), np.where(finite, fp4.unpack(rq), 0))
    for out in ("bf16", "fp16"):
        v = m.fp4_dequant_groups(q, s, group, DT[out])
        ref = torch.tensor(fp4.dequant_groups(q.cpu().numpy(), rs, group).astype(np.float32)).to(DT[out])
        assert torch.equal(torch.isnan(v).cpu(), torch.isnan(ref))
        live = ~torch.isnan(ref)
        assert torch.equal(v.cpu()[live].view(torch.int16), ref[live].view(torch.int16)), out


@pytest.mark.parametrize("fmt", ["fp32", "e8m0"])
def test_dequant_every_code_and_scale(m, fmt):
    # 16 codes under every E8M0 byte, or under fp32 scales over the whole range
    q = torch.tensor(np.tile(fp4.pack(np.arange(32) % 16), (256, 1)), device=DEV)
    if fmt == "e8m0":
        s = torch.arange(256, dtype=torch.uint8)[:, None]
    else:
        s = torch.tensor(np.ldexp(1.37, np.arange(-128, 128)).astype(np.float32))[:, None]
    for out in ("bf16", "fp16"):
        v = m.fp4_dequant_groups(q, s.to(DEV), 32, DT[out]).cpu()
        with np.errstate(over="ignore"):
            ref = torch.tensor(fp4.dequant_groups(q.cpu().numpy(), s.numpy(), 32).astype(np.float32)).to(DT[out])
        assert torch.equal(torch.isnan(v), torch.isnan(ref))
        live = ~torch.isnan(ref)
        assert torch.equal(v[live].view(torch.int16), ref[live].view(torch.int16)), out


def test_quant_strided_rows(m):
    w = _randn((20, 256), "bf16", 3)
    big = torch.full((20, 320), 99.0, dtype=torch.bfloat16, device=DEV)
    big[:, :256] = w.to(DEV)
    a, b = m.fp4_quant_groups(big[:, :256], 64), m.fp4_quant_groups(w.to(DEV), 64)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out = torch.full((20, 320), 7.0, dtype=torch.bfloat16, device=DEV)
    m.fp4_dequant_groups(*b, 64, out=out[:, :256])
    assert torch.equal(out[:, :256], m.fp4_dequant_groups(*b, 64)) and bool((out[:, 256:] == 7).all())


# ------------------------------------------------------------------ products on 4-bit weights
def _packed(shape, group, fmt, seed):
    w = _randn(shape, "bf16", seed, 0.02).float().numpy()
    q, s = fp4.quant_groups(w, group, fmt == "e8m0")
    return torch.tensor(q, device=DEV), torch.tensor(s, device=DEV), fp4.dequant_groups(q, s, group)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["fp32", "e8m0"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 40, 32), (3, 129, 96), (16, 64, 1056), (17, 100, 480), (33, 48, 1184), (70, 33, 544),
                                   (130, 272, 416)])
def test_gemm_fp4(m, dtype, fmt, group, M, N, K):
    print("fp4 gemm", dtype, fmt, group, M, N, K, flush=True)
    x = _randn((M, K), dtype, M)
    q, s, w = _packed((N, K), group, fmt, N + K)
    c = m.gemm_fp4_groupscale(x.to(DEV), q, s, group)
    xf = _f64(x)
    _close(c, xf @ w.T, np.abs(xf) @ np.abs(w).T, K, dtype, "gemm")


@pytest.mark.parametrize("M", [1, 4, 16, 20, 64])
def test_gemm_fp4_wide(m, M):
    # the widths of the linear layers; bf16, both scale formats
    for N, K, group, fmt in ((2048, 7168, 128, "fp32"), (2048, 7168, 32, "e8m0"), (576, 18432, 64, "fp32")):
        x = _randn((M, K), "bf16", M)
        q, s, w = _packed((N, K), group, fmt, N)
        c = m.gemm_fp4_groupscale(x.to(DEV), q, s, group)
        xf = _f64(x)
        _close(c, xf @ w.T, np.abs(xf) @ np.abs(w).T, K, "bf16", "gemm %dx%dx%d" % (M, N, K))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group,fmt", [(32, "fp32"), (32, "e8m0"), (64, "e8m0"), (128, "fp32")])
@pytest.mark.parametrize("N,K,rows", [(40, 4160, (2, 9, 20, 40, 64)), (7000, 4160, (2, 9, 40)), (33000, 160, (2, 9, 20, 64))])
def test_gemm_fp4_tilings(m, dtype, group, fmt, N, K, rows):
    # few, some and many columns with every row tile: each tiling of the kernel, several windows of scales
    # and scale rows that do not start on whole dwords
    q, s, w = _packed((N, K), group, fmt, N)
    for M in rows:
        print("fp4 tiling", dtype, group, fmt, N, K, M, flush=True)
        x = _randn((M, K), dtype, M)
        xf = _f64(x)
        ref, mag = xf @ w.T, np.abs(xf) @ np.abs(w).T
        _close(m.gemm_fp4_groupscale(x.to(DEV), q, s, group), ref, mag, K, dtype, "M %d" % M)
        if M > 16:
            _close(m.gemm_fp4_groupscale(x.to(DEV), q, s, group, workspace=False), ref, mag, K, dtype, "no workspace")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("spread", [12, 13, 14, 22])
def test_gemm_fp4_scales_far_apart(m, dtype, group, spread):
    # neighbouring groups' powers of two up to 2^spread apart, in some columns only; x lies in one group in
    # some rows, so that the smallest scales' products are whole results
    print("fp4 spread", dtype, group, spread, flush=True)
    for N, K, rows in ((40, 1056, (1, 7, 16, 24, 64)), (33000, 160, (2, 9, 20, 64))):
        rng = np.random.default_rng(spread)
        q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
        G = -(-K // group)
        s = np.full((N, G), 121, np.uint8)
        s[::3] = 125 - rng.choice([0, spread // 2, spread], (len(s[::3]), G)).astype(np.uint8)
        w = fp4.dequant_groups(q, s, group)
        for M in rows:
            x = _randn((M, K), dtype, M, 8.0)
            for r in range(1, M, 2):
                lo = r // 2 % G * group
                x[r, :lo], x[r, lo + group:] = 0, 0
            xf = _f64(x)
            c = m.gemm_fp4_groupscale(x.to(DEV), torch.tensor(q, device=DEV), torch.tensor(s, device=DEV), group)
            _close(c, xf @ w.T, np.abs(xf) @ np.abs(w).T, K, dtype, "%d x %d x %d" % (M, N, K))
    x[1, 5] = float("inf")  # infinite where the weight is not zero, whatever the block's other scales
    c = m.gemm_fp4_groupscale(x.to(DEV), torch.tensor(q, device=DEV), torch.tensor(s, device=DEV), group)
    assert torch.equal(c[1].isnan().cpu(), torch.tensor(w[:, 5] == 0))


def test_gemm_fp4_workspace(m):
    x, (q, s, _) = _randn((64, 8192), "bf16", 1).to(DEV), _packed((520, 8192), 64, "fp32", 2)
    n = m.gemm_fp4_groupscale_workspace(64, 520, 8192)
    assert n > 0
    want = m.gemm_fp4_groupscale(x, q, s, 64)
    for fill in (0, 255):   # its contents do not matter, and nothing is written past it
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(m.gemm_fp4_groupscale(x, q, s, 64, workspace=ws[:n]), want)
        assert bool((ws[n:] == fill).all())
    with pytest.raises(m.Moe355Error):
        m.gemm_fp4_groupscale(x, q, s, 64, workspace=ws[:n - 16])


def test_gemm_fp4_strided_and_odd_columns(m):
    for N in (1, 7, 63):
        x, (q, s, w) = _randn((5, 128), "bf16", 1), _packed((N, 128), 64, "fp32", 2)
        xb = torch.full((5, 192), float("nan"), dtype=torch.bfloat16, device=DEV)
        xb[:, :128] = x.to(DEV)
        cb = torch.full((5, N + 3), 7.0, dtype=torch.bfloat16, device=DEV)
        m.gemm_fp4_groupscale(xb[:, :128], q, s, 64, cb[:, :N])
        _close(cb[:, :N], _f64(x) @ w.T, np.abs(_f64(x)) @ np.abs(w).T, 128, "bf16")
        assert bool((cb[:, N:] == 7).all())


def test_gemm_fp4_nothing_to_do(m):
    q, s, _ = _packed((32, 64), 32, "fp32", 1)
    assert m.gemm_fp4_groupscale(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), q, s, 32).shape == (0, 32)
    z = m.gemm_fp4_groupscale(torch.empty((3, 0), dtype=torch.bfloat16, device=DEV), q[:, :0].contiguous(),
                              s[:, :0].contiguous(), 32)
    assert z.shape == (3, 32) and bool((z == 0).all())


def test_gemm_fp4_infinities_stay_in_their_rows(m):
    x = _randn((20, 256), "bf16", 5)
    q, s, w = _packed((48, 256), 32, "e8m0", 6)
    ref = m.gemm_fp4_groupscale(x.to(DEV), q, s, 32)
    x[3, 17], x[18, 200] = float("inf"), float("nan")
    got = m.gemm_fp4_groupscale(x.to(DEV), q, s, 32)
    keep = [r for r in range(20) if r not in (3, 18)]
    assert torch.equal(got[keep], ref[keep])
    assert bool(torch.isnan(got[18]).all())
    col = w[:, 17]
    assert torch.equal(got[3].isnan().cpu(), torch.tensor(col == 0))
    assert torch.equal((got[3] == float("inf")).cpu(), torch.tensor(col > 0))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,group", [("fp32", 128), ("fp32", 32), ("e8m0", 32), ("e8m0", 64)])
@pytest.mark.parametrize("counts,N,K", [([0, 1, 0, 3, 17, 0], 72, 288), ([0, 0, 5], 129, 416), ([64, 0, 130, 1], 80, 160),
                                        ([1] * 40, 32, 64), ([200, 300, 250], 144, 288)])
def test_grouped_gemm_fp4(m, dtype, fmt, group, counts, N, K):
    print("grouped fp4", dtype, fmt, group, counts[:6], N, K, flush=True)
    off, R, E = _offsets(counts), sum(counts), len(counts)
    x = _randn((R, K), dtype, R)
    q, s, w = _packed((E, N, K), group, fmt, N)
    c = m.grouped_gemm_fp4(x.to(DEV), q, s, _dev_offsets(off), group)
    ref, mag = ragged.forward(_f64(x), w, off)
    _close(c, ref, mag, K, dtype, "grouped fp4")


def test_grouped_fp4_equals_one_matrix_at_a_time(m):
    counts, N, K = [3, 0, 9, 2], 96, 640
    off = _offsets(counts)
    x = _randn((sum(counts), K), "bf16", 8).to(DEV)
    q, s, _ = _packed((4, N, K), 32, "e8m0", 9)
    c = m.grouped_gemm_fp4(x, q, s, _dev_offsets(off), 32)
    for e in (0, 2, 3):
        one = m.gemm_fp4_groupscale(x[off[e]:off[e + 1]], q[e], s[e], 32)
        assert torch.allclose(c[off[e]:off[e + 1]].float(), one.float(), rtol=2.0 ** -7, atol=1e-5)


# ------------------------------------------------------------------ ragged products
RAGGED = [([0, 1, 0, 5], 8, 8), ([3, 0, 70, 0, 64], 72, 40), ([300, 1, 0, 257], 264, 520), ([129], 1000, 136),
          ([5, 260, 512, 0, 31, 0], 512, 328), ([1] * 70, 24, 64), ([700, 900], 256, 1024)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,N,K", RAGGED)
def test_grouped_gemm_and_gradients(m, dtype, counts, N, K):
    print("ragged", dtype, counts[:6], N, K, flush=True)
    off, R, E = _offsets(counts), sum(counts), len(counts)
    x, w, dy = _randn((R, K), dtype, R), _randn((E, N, K), dtype, N, 0.05), _randn((R, N), dtype, K, 0.1)
    xd, wd, dyd, od = x.to(DEV), w.to(DEV), dy.to(DEV), _dev_offsets(off)
    ref, mag = ragged.forward(_f64(x), _f64(w), off)
    _close(m.grouped_gemm(xd, wd, od), ref, mag, K, dtype, "fwd")
    ref, mag = ragged.dgrad(_f64(dy), _f64(w), off)
    _close(m.grouped_gemm_dgrad(dyd, wd, od), ref, mag, N, dtype, "dgrad")
    ref, mag = ragged.wgrad(_f64(dy), _f64(x), off)
    for out in (dtype, "fp32"):
        dw = m.grouped_gemm_wgrad(dyd, xd, od, out_dtype=DT[out])
        _close(dw, ref, mag, max(counts), out, "wgrad " + out)
        for e in range(E):
            if counts[e] == 0:
                assert bool((dw[e] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("op,N,K", [("fwd", 5128, 136), ("fwd", 5120, 64), ("dgrad", 136, 5128), ("dgrad", 200, 5120),
                                    ("wgrad", 2600, 2568), ("wgrad", 1288, 1304)])
def test_ragged_largest_tiles(m, op, dtype, N, K):
    # enough work for the largest tile, with segments that end anywhere in one; inner sizes off its step
    counts = [700, 0, 1300, 513, 1] if op != "wgrad" else [200, 0, 97, 64, 1] * (1 if N > 2000 else 4)
    print("ragged large", op, dtype, N, K, flush=True)
    off, R, E = _offsets(counts), sum(counts), len(counts)
    x, w, dy = _randn((R, K), dtype, R), _randn((E, N, K), dtype, N, 0.05), _randn((R, N), dtype, K, 0.1)
    od = _dev_offsets(off)
    if op == "fwd":
        got, (ref, mag), n = m.grouped_gemm(x.to(DEV), w.to(DEV), od), ragged.forward(_f64(x), _f64(w), off), K
    elif op == "dgrad":
        got, (ref, mag), n = m.grouped_gemm_dgrad(dy.to(DEV), w.to(DEV), od), ragged.dgrad(_f64(dy), _f64(w), off), N
    else:
        got, (ref, mag), n = m.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), od), ragged.wgrad(_f64(dy), _f64(x), off), max(counts)
    _close(got, ref, mag, n, dtype, op)


def test_one_expert_with_most_rows(m):
    # few rows an expert on average, nearly all of them in one: its passes
    counts, N, K = [0] * 9 + [150] + [1] * 30, 264, 320
    off, R = _offsets(counts), sum(counts)
    x, w = _randn((R, K), "bf16", 1), _randn((40, N, K), "bf16", 2, 0.05)
    ref, mag = ragged.forward(_f64(x), _f64(w), off)
    _close(m.grouped_gemm(x.to(DEV), w.to(DEV), _dev_offsets(off)), ref, mag, K, "bf16", "16-bit weights")
    q, s, wf = _packed((40, N, K), 32, "e8m0", 3)
    ref, mag = ragged.forward(_f64(x), wf, off)
    _close(m.grouped_gemm_fp4(x.to(DEV), q, s, _dev_offsets(off), 32), ref, mag, K, "bf16", "4-bit weights")


def test_ragged_strided_rows(m):
    counts, N, K = [30, 0, 41], 136, 72
    off, R = _offsets(counts), sum(counts)
    x, w, dy = _randn((R, K), "bf16", 1), _randn((3, N, K), "bf16", 2), _randn((R, N), "bf16", 3)

    def wide(t, pad):
        b = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
        b[:, :t.shape[1]] = t.to(DEV)
        return b[:, :t.shape[1]]

    xs, dys, wd, od = wide(x, 56), wide(dy, 8), w.to(DEV), _dev_offsets(off)
    y = torch.full((R, N + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    dx = torch.full((R, K + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    m.grouped_gemm(xs, wd, od, y[:, :N])
    m.grouped_gemm_dgrad(dys, wd, od, dx[:, :K])
    assert torch.equal(y[:, :N], m.grouped_gemm(x.to(DEV), wd, od)) and bool((y[:, N:] == 7).all())
    assert torch.equal(dx[:, :K], m.grouped_gemm_dgrad(dy.to(DEV), wd, od)) and bool((dx[:, K:] == 7).all())
    assert torch.equal(m.grouped_gemm_wgrad(dys, xs, od), m.grouped_gemm_wgrad(dy.to(DEV), x.to(DEV), od))


def test_ragged_neighbours_infinities_stay_out(m):
    # a row of NaN and infinities in each neighbour of expert 1, next to its first and last rows
    counts, N, K = [5, 61, 9], 72, 136
    off, R = _offsets(counts), sum(counts)
    x, w, dy = _randn((R, K), "bf16", 1), _randn((3, N, K), "bf16", 2), _randn((R, N), "bf16", 3)
    od, wd = _dev_offsets(off), w.to(DEV)

    def all_three(x, dy):
        x, dy = x.to(DEV), dy.to(DEV)
        return m.grouped_gemm(x, wd, od), m.grouped_gemm_dgrad(dy, wd, od), m.grouped_gemm_wgrad(dy, x, od)

    want = all_three(x, dy)
    x[4], x[66], dy[4], dy[66] = float("nan"), float("inf"), float("inf"), float("nan")
    got = all_three(x, dy)
    keep = [r for r in range(R) if r not in (4, 66)]
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
    assert torch.equal(got[2][1], want[2][1])
    assert not bool(torch.isfinite(got[0][[4, 66]]).any())
    assert not bool(torch.isfinite(got[2][[0, 2]]).any())


def test_ragged_nothing_to_do(m):
    w = _randn((3, 16, 24), "bf16", 1).to(DEV)
    od = _dev_offsets([0, 0, 0, 0])
    e = lambda c: torch.empty((0, c), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    assert m.grouped_gemm(e(24), w, od).shape == (0, 16)
    assert m.grouped_gemm_dgrad(e(16), w, od).shape == (0, 24)
    dw = torch.full((3, 16, 24), 7.0, dtype=torch.float32, device=DEV)
    assert bool((m.grouped_gemm_wgrad(e(16), e(24), od, dw) == 0).all())
    # no inner dimension: zeros
    x = torch.empty((5, 0), dtype=torch.bfloat16, device=DEV)
    assert bool((m.grouped_gemm(x, torch.empty((1, 16, 0), dtype=torch.bfloat16, device=DEV), _dev_offsets([0, 5])) == 0).all())


def test_rows_outside_segments_are_left_alone(m):
    off, R, N, K = [2, 10, 10, 25], 40, 40, 64
    x, w, od = _randn((R, K), "bf16", 1).to(DEV), _randn((3, N, K), "bf16", 2).to(DEV), _dev_offsets(off)
    q, s, _ = _packed((3, N, K), 32, "fp32", 3)
    outside = list(range(2)) + list(range(25, 40))
    for call in (lambda c: m.grouped_gemm(x, w, od, c), lambda c: m.grouped_gemm_fp4(x, q, s, od, 32, c)):
        c = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
        call(c)
        assert bool((c[outside] == 7).all()) and not bool((c[2:25] == 7).all(dim=1).any())


@pytest.mark.parametrize("off", [[-5, 3, 900, 20], [0, 30, 10, 40], [50, 60, 70, 80]])
def test_offsets_out_of_range_touch_nothing_outside(m, off):
    # the kernels cut offsets to [0, R] and decreasing segments to nothing: the guard bands stay
    R, N, K, E = 40, 72, 96, 3
    od = _dev_offsets(off)
    q, s, _ = _packed((E, N, K), 32, "fp32", 3)
    w = _randn((E, N, K), "bf16", 2).to(DEV)

    def banded(rows, cols, fill=7.0):
        b = torch.full((rows + 64, cols), fill, dtype=torch.bfloat16, device=DEV)
        return b, b[32:32 + rows]

    xb, x = banded(R, K)
    dyb, dy = banded(R, N)
    x.copy_(_randn((R, K), "bf16", 1))
    dy.copy_(_randn((R, N), "bf16", 4))
    for cols, call in ((N, lambda c: m.grouped_gemm(x, w, od, c)), (K, lambda c: m.grouped_gemm_dgrad(dy, w, od, c)),
                       (N, lambda c: m.grouped_gemm_fp4(x, q, s, od, 32, c))):
        b, c = banded(R, cols)
        call(c)
        assert bool((b[:32] == 7).all()) and bool((b[32 + R:] == 7).all())
    flat = torch.full((E * N + 64, K), 7.0, dtype=torch.bfloat16, device=DEV)
    m.grouped_gemm_wgrad(dy, x, od, flat[32:32 + E * N].view(E, N, K))
    assert bool((flat[:32] == 7).all()) and bool((flat[32 + E * N:] == 7).all())


def test_gradient_against_differences(m):
    # the loss sum(y * g) is linear in x and in w: its central difference in 64 bits is exact, and the
    # gradients' inner products with a direction match it within the gradients' rounding
    counts, N, K = [7, 0, 33], 40, 56
    off, R = _offsets(counts), sum(counts)
    x, w, g = _randn((R, K), "bf16", 1), _randn((3, N, K), "bf16", 2), _randn((R, N), "bf16", 3)
    tx, tw = x.to(DEV).requires_grad_(), w.to(DEV).requires_grad_()
    m.grouped_linear(tx, tw, _dev_offsets(off)).backward(g.to(DEV))
    loss = lambda a, b: float((ragged.forward(a, b, off)[0] * _f64(g)).sum())  # noqa: E731
    rng = np.random.default_rng(0)
    for grad, of in ((tx.grad, "x"), (tw.grad, "w")):
        d = rng.normal(size=grad.shape)
        X, W, h = _f64(x), _f64(w), 0.5
        diff = (loss(X + h * d, W) - loss(X - h * d, W)) if of == "x" else (loss(X, W + h * d) - loss(X, W - h * d))
        tol = 2.0 ** -8 * float(np.abs(_f64(grad) * d).sum())
        assert abs(float((_f64(grad) * d).sum()) - diff) <= tol, of


def test_grouped_linear_needs_only_what_is_asked(m):
    x, w, od = _randn((6, 16), "bf16", 1).to(DEV), _randn((2, 24, 16), "bf16", 2).to(DEV), _dev_offsets([0, 2, 6])
    a = x.clone().requires_grad_()
    m.grouped_linear(a, w, od).sum().backward()
    assert a.grad is not None and w.grad is None
    b = w.clone().requires_grad_()
    m.grouped_linear(x, b, od).sum().backward()
    assert torch.equal(b.grad, m.grouped_gemm_wgrad(torch.ones((6, 24), dtype=torch.bfloat16, device=DEV), x, od))


# ------------------------------------------------------------------ use
def test_results_repeat_and_follow_the_stream(m):
    counts, N, K = [40, 0, 300, 7], 520, 1160
    off, R = _offsets(counts), sum(counts)
    x, w, dy = (_randn((R, K), "bf16", 1).to(DEV), _randn((4, N, K), "bf16", 2).to(DEV), _randn((R, N), "bf16", 3).to(DEV))
    q, s, _ = _packed((4, N, 1152), 128, "fp32", 4)
    xq, od = x[:, :1152], _dev_offsets(off)
    calls = [lambda: m.grouped_gemm(x, w, od), lambda: m.grouped_gemm_dgrad(dy, w, od),
             lambda: m.grouped_gemm_wgrad(dy, x, od, out_dtype=torch.float32), lambda: m.grouped_gemm_fp4(xq, q, s, od),
             lambda: m.gemm_fp4_groupscale(xq[:50], q[0], s[0])]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = [c() for c in calls]
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_graph_replays_match_eager(m):
    counts, N, K = [3, 0, 20, 1], 264, 384
    off, R = _offsets(counts), sum(counts)
    x, w, dy = (_randn((R, K), "bf16", 1).to(DEV), _randn((4, N, K), "bf16", 2).to(DEV), _randn((R, N), "bf16", 3).to(DEV))
    q, s = m.fp4_quant_groups(w, 64)
    od = _dev_offsets(off)

    def step():
        return [m.grouped_gemm(x, w, od), m.grouped_gemm_dgrad(dy, w, od), m.grouped_gemm_wgrad(dy, x, od),
                m.grouped_gemm_fp4(x, q, s, od, 64), m.gemm_fp4_groupscale(x, q[1], s[1], 64),
                m.fp4_dequant_groups(*m.fp4_quant_groups(w, 64), 64)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(_randn((R, K), "bf16", 10 + i))
        dy.copy_(_randn((R, N), "bf16", 20 + i))
        od.copy_(torch.tensor(_offsets([[3, 0, 20, 1], [0, 0, 24, 0], [24, 0, 0, 0], [6, 6, 6, 6]][i]), dtype=torch.int32))
        torch.cuda.synchronize()
        want = step()
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


def test_weights_beyond_32_bit_offsets(m):
    # 16-bit weights of 2^32 + elements and codes of 2^32 + bytes: the last expert's products and gradient
    N, K, E = 4096, 8192, 129
    print("large offsets", flush=True)
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    w[-1] = torch.randn((N, K), generator=g, device=DEV) * 0.02
    x = torch.randn((40, K), generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn((40, N), generator=g, device=DEV).to(torch.bfloat16)
    od = _dev_offsets([0] * E + [40])
    ref, mag = ragged.forward(_f64(x), _f64(w[-1:]), [0, 40])
    _close(m.grouped_gemm(x, w, od), ref, mag, K, "bf16", "fwd")
    ref, mag = ragged.dgrad(_f64(dy), _f64(w[-1:]), [0, 40])
    _close(m.grouped_gemm_dgrad(dy, w, od), ref, mag, N, "bf16", "dgrad")
    dw = m.grouped_gemm_wgrad(dy, x, od)
    ref, mag = ragged.wgrad(_f64(dy), _f64(x), [0, 40])
    _close(dw[-1:], ref, mag, 40, "bf16", "wgrad")
    assert bool((dw[:-1] == 0).all())
    del w, dw
    E = 257
    q = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.ones((E, N, K // 128), dtype=torch.float32, device=DEV)
    q[-1] = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    od = _dev_offsets([0] * E + [40])
    wq = fp4.dequant_groups(q[-1].cpu().numpy(), s[-1].cpu().numpy(), 128)
    ref, mag = ragged.forward(_f64(x), wq[None], [0, 40])
    _close(m.grouped_gemm_fp4(x, q, s, od), ref, mag, K, "bf16", "fp4")
    big = m.fp4_dequant_groups(q, s)
    assert torch.equal(big[-1], m.fp4_dequant_groups(q[-1], s[-1])) and bool((big[-2] == 0).all())
    q2, s2 = m.fp4_quant_groups(big)
    assert torch.equal(s2[-1], m.fp4_quant_groups(big[-1])[1]) and torch.equal(q2[-1], m.fp4_quant_groups(big[-1])[0])
    del q, s, big, q2, s2
    torch.cuda.empty_cache()


def test_binding_refuses(m):
    x, w, od = _randn((6, 16), "bf16", 1).to(DEV), _randn((2, 24, 16), "bf16", 2).to(DEV), _dev_offsets([0, 2, 6])
    q, s = m.fp4_quant_groups(_randn((24, 64), "bf16", 3).to(DEV), 32)
    x4 = _randn((6, 64), "bf16", 4).to(DEV)
    bad = [lambda: m.grouped_gemm(x.float(), w, od), lambda: m.grouped_gemm(x, w.half(), od),
           lambda: m.grouped_gemm(x, w, od.long()), lambda: m.grouped_gemm(x, w, od[:2]), lambda: m.grouped_gemm(x.t(), w, od),
           lambda: m.grouped_gemm(x, w, od.cpu()), lambda: m.grouped_gemm(x, w, od, x), lambda: m.grouped_gemm_dgrad(x, w, od),
           lambda: m.grouped_gemm_wgrad(x, x, od, out_dtype=torch.float16), lambda: m.grouped_gemm_wgrad(x, x[:3], od),
           lambda: m.gemm_fp4_groupscale(x, q, s, 32), lambda: m.gemm_fp4_groupscale(x4, q, s, 64),
           lambda: m.gemm_fp4_groupscale(x4, q, s, 48), lambda: m.gemm_fp4_groupscale(x4, q, s.half(), 32),
           lambda: m.gemm_fp4_groupscale(x4.cpu(), q, s, 32), lambda: m.fp4_quant_groups(x4, 32, "int8"),
           lambda: m.fp4_quant_groups(x4.float(), 32), lambda: m.fp4_dequant_groups(q, s, 32, torch.float32),
           lambda: m.fp4_dequant_groups(q, s, 64)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was accepted" % i)
    for code, f in ((-2, lambda: m.fp4_quant_groups(_randn((4, 48), "bf16", 1).to(DEV), 32)),
                    (-3, lambda: m.gemm_fp4_groupscale(_randn((4, 72), "bf16", 1).to(DEV)[:, 4:68], q, s, 32)),
                    (-2, lambda: m.grouped_gemm(x[:, :12], w[:, :, :12].contiguous(), od)),
                    (-3, lambda: m.grouped_gemm(_randn((6, 20), "bf16", 1).to(DEV)[:, :16], w, od))):
        with pytest.raises(m.Moe355Error) as err:
            f()
        assert err.value.code == code


# ------------------------------------------------------------------ together
def _layer64(x, ids, weights, w1, w2, s1, s2):
    """The example's layer in 64 bits, and a bound of what bf16 between the products costs: with u = 2^-8,
    gate, up and h are each rounded once (SiLU's relative slope stays below 1.3 + |gate|, taken as it
    is), y and the shared product once more."""
    silu = lambda v: v / (1 + np.exp(-v))  # noqa: E731
    u = 2.0 ** -8

    def gated(rows, a, b):
        z, zm = rows @ a.T, np.abs(rows) @ np.abs(a).T
        i = a.shape[0] // 2
        gate, up = z[:, :i], z[:, i:]
        h = silu(gate) * up
        dg, du = u * np.abs(gate) + 1e-5 * zm[:, :i], u * np.abs(up) + 1e-5 * zm[:, i:]
        dh = 1.1 * dg * (np.abs(up) + du) + np.abs(silu(gate)) * du    # |SiLU'| < 1.1
        dh = dh + u * (np.abs(h) + dh)
        y, ym = h @ b.T, np.abs(h) @ np.abs(b).T
        dy = dh @ np.abs(b).T + 1e-5 * ym
        return y, dy + u * (np.abs(y) + dy)

    out, tol = gated(x, s1, s2)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            y, d = gated(x[t:t + 1], w1[e], w2[e])
            out[t] += weights[t, j] * y[0]
            tol[t] += abs(weights[t, j]) * d[0] * 1.001
    return out, tol + 1e-5 * np.abs(out) + 1e-6


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T", [1, 40])
def test_example_layer(m, packed, T):
    from fp8_block_scaled_grouped_amd.examples.ragged_experts import RaggedExperts
    layer = RaggedExperts(H=64, I=96, E=8, n_group=4, topk_group=2, topk=3, device=DEV, seed=3)
    x, logits = _randn((T, 64), "bf16", T).to(DEV), torch.randn((T, 8), generator=torch.Generator().manual_seed(T)).to(DEV)
    names = ("w1", "w2", "s1", "s2")
    if packed:
        layer.pack(32, "e8m0")
        ws = [fp4.dequant_groups(q.cpu().numpy(), s.cpu().numpy(), 32) for q, s in (layer.packed[n] for n in names)]
    else:
        ws = [_f64(getattr(layer, n).to(torch.bfloat16)) for n in names]
    weights, ids = m.grouped_topk(logits, layer.bias, *layer.route)
    ref, tol = _layer64(_f64(x), ids.cpu().numpy(), _f64(weights), *ws)
    err = np.abs(_f64(layer(x, logits)) - ref)
    assert (err <= tol).all(), float((err / tol).max())


def test_example_trains_and_packs(m):
    from fp8_block_scaled_grouped_amd.examples.ragged_experts import RaggedExperts, train
    shape = dict(H=128, I=64, E=8, n_group=4, topk_group=2, topk=2, device=DEV)
    layer, teacher = RaggedExperts(**shape, seed=1), RaggedExperts(**shape, seed=2)
    x = _randn((256, 128), "bf16", 1).to(DEV)
    logits = torch.randn((256, 8), generator=torch.Generator().manual_seed(2)).to(DEV)
    losses = train(layer, teacher, x, logits, 15).cpu()
    assert bool(torch.isfinite(losses).all()) and float(losses[-1]) < 0.9 * float(losses[0])
    assert all(p.grad is not None and bool(torch.isfinite(p.grad).all()) for p in layer.parameters())
    before = layer(x, logits).detach()
    after = layer.pack()(x, logits)
    # 4-bit weights: each product's weights are off by at most half a step of e2m1, 1/6 of their value at worst
    assert float((after - before).norm() / before.norm()) < 0.5
