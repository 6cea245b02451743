"""FP8 operands and ragged expert products at the ends of their ranges, against the 64-bit oracle; tolerances as in
test_gpu_fp8_ragged.py."""
import numpy as np
import pytest
import torch

from oracle import fp8_ragged as o, ragged
from tests import fp8_ragged_tilings as t
from tests.test_gpu_fp8_ragged import DEV, DT, _close, _dev, _offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import fp8_block_scaled_grouped_amd as mod
    mod.lib()
    return mod


# ------------------------------------------------------------------ fp32 scales
# (binary exponents of x's scales, of w's, smallest code, codes): products of two scales below 2^-126 under sums of 2^23 and more, close to
# 2^128 over sums of 2^-11 and less, and ordinary ones
SCALES = [((-74, -72), (-74, -72), 0x78, 7), ((-140, -128), (-20, -4), 0x78, 7), ((-20, -4), (-140, -128), 0x78, 7),
          ((64, 66), (56, 59), 0x01, 2), ((100, 104), (18, 21), 0x01, 2), ((-3, 3), (-3, 3), 0x30, 16)]
ONE_OF_EACH = [t.PRODUCTS[i] for i in (1, 6, 9, 11)]


@pytest.mark.parametrize("ex,ew,code,codes", SCALES)
@pytest.mark.parametrize("counts,N,K", ONE_OF_EACH + [([3], 8, 16)])
def test_products_of_scales_at_the_ends_of_fp32(m, counts, N, K, ex, ew, code, codes):
    """Two scales are multiplied first, in fp32: below 2^-126 the product is off by up to 2^-150, so a block by that times its sum of
    products of codes; each addition in that range by up to 2^-150 as well.  Codes of one sign, so sums are not small by chance."""
    print("scales", counts[:4], N, K, ex, ew, flush=True)
    E, R, KB, NB, g = len(counts), sum(counts), -(-K // 128), -(-N // 128), np.random.default_rng(N + K)
    assert len({t.tile("fwd", sum(c), len(c), n, k) for c, n, k in ONE_OF_EACH}) == 4
    off = _offsets(counts)
    scale = lambda a, shape: np.ldexp(g.uniform(1, 2, shape), g.integers(a[0], a[1] + 1, shape)).astype(np.float32)
    xs, ws = scale(ex, (R, KB)), scale(ew, (E, NB, KB))
    xq, wq = (g.integers(code, code + codes, shape, dtype=np.uint8) for shape in ((R, K), (E, N, K)))
    xs[0, 0], xq[R - 1] = 0, 0               # a block with a scale of zero, a row of zeros
    y = m.grouped_gemm_fp8(*(torch.tensor(v, device=DEV) for v in (xq, xs, wq, ws)), _dev(off)).cpu()
    ref, mag = ragged.forward(o.values(xq, xs, 1), o.values(wq, ws, 128), off)
    sums = ragged.forward(o.fp8.decode(xq), o.fp8.decode(wq), off)[1]
    each = o.each(xs, 1, R, K)
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if a < b:
            unit = o.unit_bound(xq[a:b], each[a:b], wq[e], o.each(ws[e], 128, N, K)) + (sums[a:b] + KB) * 2.0 ** -150
            _close(y[a:b], ref[a:b], mag[a:b], K, "bf16", "y of expert %d" % e, unit)
    assert (y[R - 1] == 0).all()


def test_scales_of_zero_infinity_and_nan(m):
    """Zero wins over any finite scale, infinities and NaN come through."""
    K, N = 128, 16
    code = torch.full((6, K), 0x7e, dtype=torch.uint8, device=DEV)
    xs = torch.tensor([0.0, 1.0, float("inf"), float("nan"), -2.0, -float("inf")], device=DEV)[:, None]
    for ws, finite in ((2.0 ** 126, False), (1.0, True), (2.0 ** -126, True)):
        y = m.grouped_gemm_fp8(code, xs, code[:1].expand(1, N, K).contiguous(), torch.full((1, 1, 1), ws, device=DEV), _dev([0, 6])).float()
        assert (y[0] == 0).all() and (y[2] == float("inf")).all() and y[3].isnan().all() and (y[5] == -float("inf")).all()
        assert torch.isfinite(y[1]).all() == finite and torch.isfinite(y[4]).all() == finite and (y[4] < 0).all()


def test_sizes_that_32_bits_would_cut_are_refused(m):
    """The library's sizes are C ints: 2^32 + n must not pass for n."""
    row, off = torch.zeros((1, 16), dtype=torch.bfloat16, device=DEV), _dev([0, 16])
    z = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=DEV)
    many = row.expand(2 ** 32 + 16, 16)
    w = torch.empty((1, 1, 2 ** 32 + 128), dtype=torch.bfloat16, device=DEV)
    for call in (lambda: m.fp8_quant_ragged(many), lambda: m.fp8_quant_ragged(many, off), lambda: m.fp8_quant_128x128(w),
                 lambda: m.grouped_linear_fp8(many, torch.zeros((1, 16, 16), dtype=torch.bfloat16, device=DEV), off),
                 lambda: m.grouped_gemm_fp8_wgrad(z(1, 16, 128), z(1, 16), z(1, 16, 128), z(1, 16), off, 2 ** 32 + 16)):
        with pytest.raises(ValueError, match=r"below 2\^31"):
            call()


# ------------------------------------------------------------------ offsets past 4 GiB
ONE = 0x38                                                                # the code of 1.0


def _bytes(shape, value):
    return torch.full(shape, value, dtype=torch.uint8, device=DEV)


def test_outputs_past_two_to_the_32_bytes(m):
    E, N, K = 3, 1 << 15, 16
    R = (1 << 32) // (2 * N) + 300
    off = [0, R - 260, R - 130, R]
    x8 = _bytes((R, K), 0)
    x8[R - 260:] = ONE
    ws = _bytes((E, N // 128, 1), 127)
    ws[2] = 128
    y = m.grouped_gemm_fp8(x8, _bytes((1, 1), 127).expand(R, 1), _bytes((E, N, K), ONE), ws, _dev(off))
    assert not y[:R - 260].any() and (y[R - 260:R - 130] == K).all() and (y[R - 130:] == 2 * K).all()


def test_weights_past_two_to_the_32_bytes(m):
    """Weights of 4.3 GB: quantised, both ways, and the last two experts multiplied, by two tiles."""
    E, N, K = 66, 1 << 12, 1 << 14
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEV)
    w[E - 1], w[E - 2, -1] = 1.0, 2.0
    q, s, qt, ts = m.fp8_quant_128x128(w, transposed=True)
    del w
    # the smallest power of two that keeps 1 (2) in +-448 is 2^-8 (2^-7), 256 of which is code 0x78
    assert (q[E - 1] == 0x78).all() and (q[E - 2, -1] == 0x78).all() and not q[:E - 2].any() and not q[E - 2, :-1].any()
    assert (qt[E - 1] == 0x78).all() and (qt[E - 2, :, -1] == 0x78).all() and not qt[:E - 2].any() and not qt[E - 2, :, :-1].any()
    assert (s[E - 1] == 119).all() and (ts[E - 1] == 119).all() and (s[:E - 2] == 127).all() and (ts[:E - 2] == 127).all()
    assert (s[E - 2, -1] == 120).all() and (s[E - 2, :-1] == 127).all() and (ts[E - 2, :, -1] == 120).all() and (ts[E - 2, :, :-1] == 127).all()
    del qt
    for n in (3, 3000):
        off = [0] * (E - 2) + [0, n, 2 * n]
        y = m.grouped_gemm_fp8(_bytes((2 * n, K), ONE), _bytes((1, 1), 127).expand(2 * n, K // 128), q, s, _dev(off))
        assert not y[:n, :-1].any() and (y[:n, -1] == 2 * K).all() and (y[n:] == K).all()


@pytest.mark.parametrize("N,K", [(16, 1 << 15), (1 << 15, 16)])
def test_codes_and_blocks_past_two_to_the_32_bytes(m, N, K):
    """Rows' codes and transposed blocks of 4.3 GB, written and multiplied: those of x, and those of dy."""
    E, wide = 3, 1 << 15
    R = (1 << 32) // wide + 300
    off = [0, R - 260, R - 130, R]
    t = torch.zeros((R, wide), dtype=torch.bfloat16, device=DEV)
    t[R - 260:] = 1
    q, s, qt, ts = m.fp8_quant_ragged(t, _dev(off))
    del t
    assert (q[R - 260:] == 0x78).all() and not q[:R - 260].any() and (s[R - 260:] == 119).all() and (s[:R - 260] == 127).all()
    b = [off[e] // 128 + e for e in (1, 2)]                                # blocks of the last experts: 128 rows and 2
    for first in b:
        assert (qt[first] == 0x78).all() and (qt[first + 1, :, :2] == 0x78).all() and not qt[first + 1, :, 2:].any()
        assert (ts[first:first + 2] == 119).all()
    assert not qt[:off[1] // 128].any() and (ts[:off[1] // 128] == 127).all()
    del q, s
    _, _, ot, ots = m.fp8_quant_ragged(torch.ones((R, 16), dtype=torch.bfloat16, device=DEV), _dev(off), rows=False)
    args = (qt, ts, ot, ots) if N > K else (ot, ots, qt, ts)
    dw = m.grouped_gemm_fp8_wgrad(*args, _dev(off), R)
    assert not dw[0].any() and (dw[1:] == 130).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_gradients_of_weights_past_two_to_the_32_bytes(m, out):
    E, N, K, R = 3, 1 << 15, 1 << 15, 130
    off = _dev([0, 1, 1, R])
    dy, x = (torch.ones((R, n), dtype=torch.bfloat16, device=DEV) for n in (N, K))
    dy[R - 1, -1] = 3
    (dyt, dys), (xt, xs) = (m.fp8_quant_ragged(v, off, rows=False)[2:] for v in (dy, x))
    dw = m.grouped_gemm_fp8_wgrad(dyt, dys, xt, xs, off, R, out_dtype=out)
    assert (dw[0] == 1).all() and not dw[1].any() and (dw[2, :-1] == R - 1).all()
    assert (dw[2, -1] == torch.tensor(R + 1.0).to(out)).all()


# ------------------------------------------------------------------ every value under every scale
def _bits(first, end, dt):
    return torch.arange(first, end, dtype=torch.int32).to(torch.int16).view(dt)


def _blocks(dt, n):
    """Blocks of n values whose first is the largest magnitude with an E8M0 byte, the others all values up to it with both signs, and the
    byte of each block: every pair of a value and a byte that quantisation can bring together."""
    mags = _bits(0, 0x7f80 if dt == torch.bfloat16 else 0x7c00, dt)
    byte = torch.from_numpy(o.e8m0_byte(mags.double().numpy())).long()
    blocks, bytes_ = [], []
    for c in byte[1:].unique().tolist():                                   # (zero has a byte of its own, which others have too)
        last = int((byte[1:] == c).nonzero().max()) + 1                    # magnitudes ascend with their bits
        some = torch.cat([mags[:last + 1], -mags[:last + 1]])
        some = torch.nn.functional.pad(some, (0, -some.numel() % (n - 1))).view(-1, n - 1)
        blocks.append(torch.cat([mags[last].expand(some.shape[0], 1), some], 1))
        bytes_ += [c] * some.shape[0]
    return torch.cat(blocks), np.array(bytes_, np.uint8), byte


@pytest.mark.parametrize("dtype,first,last", [("bf16", 0, 247), ("fp16", 95, 135)])
def test_every_value_under_every_scale_that_its_block_can_have(m, dtype, first, last):
    """All bytes from the smallest subnormal's (bf16: 0, where the scale is kept at 2^-127) to the largest finite value's."""
    dt = DT[dtype]
    x, c, byte = _blocks(dt, 128)
    assert set(c.tolist()) == set(range(first, last + 1))
    ref = o.fp8.encode(x.double().numpy() / o.e8m0_value(c)[:, None])
    q, s, _, _ = m.fp8_quant_ragged(x.to(DEV), columns=False)
    assert (s[:, 0].cpu().numpy() == c).all() and (q.cpu().numpy() == ref).all()
    xt = x.t()[:, :x.shape[0] // 8 * 8].contiguous()                       # the same blocks as columns of 128 rows
    _, _, qt, ts = m.fp8_quant_ragged(xt.to(DEV), _dev([0, 128]), rows=False)
    n = xt.shape[1]
    assert (ts[0].cpu().numpy() == c[:n]).all() and (qt[0].cpu().numpy() == ref[:n]).all()
    w, c, _ = _blocks(dt, 128 * 128)
    q, s, qt, ts = m.fp8_quant_128x128(w.view(-1, 128, 128).to(DEV), transposed=True)
    ref = o.fp8.encode(w.double().numpy() / o.e8m0_value(c)[:, None]).reshape(-1, 128, 128)
    assert (s.flatten().cpu().numpy() == c).all() and (q.cpu().numpy() == ref).all()
    assert torch.equal(qt, q.transpose(1, 2)) and torch.equal(ts, s)


@pytest.mark.parametrize("dtype,end", [("bf16", 0x7f80), ("fp16", 0x7c00)])
def test_every_magnitude_as_the_largest_of_a_block(m, dtype, end):
    """The bytes of blocks whose largest magnitude is each finite value, and 255 for infinity and every NaN, alone in a block of zeros."""
    v = _bits(0, 0x8000, DT[dtype])
    want = np.where(np.arange(0x8000) < end, o.e8m0_byte(v.double().nan_to_num(0).numpy()), 255)
    for sign in (1, -1):
        x = torch.zeros((0x8000, 128), dtype=DT[dtype])
        x[:, 77] = v if sign > 0 else (v.view(torch.int16) | -0x8000).view(DT[dtype])
        _, s, _, ts = m.fp8_quant_ragged(x.t().contiguous().to(DEV), _dev([0, 128]))
        assert (ts[0].cpu().numpy() == want).all()
        _, s, _, _ = m.fp8_quant_ragged(x.to(DEV), columns=False)
        assert (s[:, 0].cpu().numpy() == want).all()
