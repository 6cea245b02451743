"""Every kernel of the 4-bit and ragged products against the formulas in 64 bits.

Inputs whose sums are exact: x and dy are small whole numbers, weights multiples of 1/4 with powers of two as scales, so
every partial sum is a multiple of 2^-2 below 2^21 and fp32 holds it in any order.  The output is then the rounded exact
value, and nothing else: a k, a row or a scale that is lost or taken twice shows, at any length.

Sums of normal numbers over a long K are compared by their root mean square error.  Rounding the output leaves half a
unit in the last place over sqrt(3) (uniform), R over all outputs; the sum takes a step per 32 k, each off by at most
2^-23 of a partial sum, whose mean square is below the output's.  The bound is 1.1 R + (K / 32 + 8) 2^-23 RMS(output).
"""
import numpy as np
import pytest
import torch

from oracle import fp4, ragged
from tests import fp4_ragged_tilings as t

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def m():
    import fp8_block_scaled_grouped_amd as mod
    mod.lib()
    return mod


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _whole(shape, dtype, seed):
    return torch.randint(-4, 5, shape, generator=_gen(seed), device=DEV).to(DT[dtype])


def _weights4(shape, group, fmt, seed):
    """Codes and power-of-two scales of weights `shape`, each scale twice, once or half."""
    g, (*lead, K) = _gen(seed), shape
    q = torch.randint(0, 256, (*lead, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randint(126, 129, (*lead, -(-K // group)), generator=g, device=DEV)
    return q, s.to(torch.uint8) if fmt == "e8m0" else torch.exp2((s - 127).float())


def _values(q, s, group):
    """fp64 weights on the GPU."""
    levels = torch.tensor(np.concatenate([fp4.LEVELS, -fp4.LEVELS]), device=DEV)
    v = torch.stack([levels[(q & 15).long()], levels[(q >> 4).long()]], -1).flatten(-2)
    s = torch.exp2(s.double() - 127) if s.dtype == torch.uint8 else s.double()
    return v * s.repeat_interleave(group, -1)[..., :v.shape[-1]]


def _offsets(counts):
    return [0] + np.cumsum(counts).tolist()


def _same(got, ref, what):
    want = ref.to(got.dtype)  # exact in fp32, so rounded once
    bad = got != want
    assert not bool(bad.any()), "%s: %d of %d differ, first at %s: %r, not %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float(got[bad][0]), float(want[bad][0]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,group", t.FORMATS)
def test_linear(m, dtype, fmt, group):
    have = None
    for M, N, K in t.LINEAR:
        if have != (N, K):
            have, (q, s) = (N, K), _weights4((N, K), group, fmt, N + K)
            w = _values(q, s, group).t()
        tiling = t.skinny(fmt, group, dtype == "fp16", M, 0, N, K)
        print("4-bit linear", dtype, fmt, group, M, N, K, tiling, flush=True)
        x = _whole((M, K), dtype, M)
        for workspace in (None, False):
            _same(m.gemm_fp4_groupscale(x, q, s, group, workspace=workspace), x.double() @ w, "%d x %d x %d, %s" % (M, N, K, tiling))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,group", t.FORMATS)
def test_experts(m, dtype, fmt, group):
    for counts, N, K in t.EXPERTS:
        off, E = _offsets(counts), len(counts)
        tiling = t.skinny(fmt, group, dtype == "fp16", off[-1], E, N, K)
        print("4-bit experts", dtype, fmt, group, off[-1], E, N, K, tiling, flush=True)
        q, s = _weights4((E, N, K), group, fmt, N + K)
        x = _whole((off[-1], K), dtype, E)
        c = m.grouped_gemm_fp4(x, q, s, torch.tensor(off, dtype=torch.int32, device=DEV), group)
        for e in range(E):
            a, b = off[e], off[e + 1]
            if b > a:
                _same(c[a:b], x[a:b].double() @ _values(q[e], s[e], group).t(), "expert %d of %d x %d x %d, %s" % (e, E, N, K, tiling))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("op,counts,N,K", [("fwd", *c) for c in t.WEIGHTS16] + t.RAGGED)
def test_ragged(m, dtype, op, counts, N, K):
    off, E, R = _offsets(counts), len(counts), sum(counts)
    print("ragged", op, dtype, R, E, N, K, t.ragged(op, R, E, N, K), flush=True)
    x, w, dy = _whole((R, K), dtype, 1), _whole((E, N, K), dtype, 2), _whole((R, N), dtype, 3)
    w = w / 4 if op != "wgrad" else w
    od = torch.tensor(off, dtype=torch.int32, device=DEV)
    if op == "wgrad":
        got = {"fp32": m.grouped_gemm_wgrad(dy, x, od, out_dtype=torch.float32), dtype: m.grouped_gemm_wgrad(dy, x, od)}
    else:
        got = m.grouped_gemm(x, w, od) if op == "fwd" else m.grouped_gemm_dgrad(dy, w, od)
    for e in range(E):
        a, b = off[e], off[e + 1]
        if op == "wgrad":
            for k, v in got.items():
                _same(v[e], dy[a:b].double().t().contiguous() @ x[a:b].double(), "%s of expert %d" % (k, e))
        elif b > a:
            ref = x[a:b].double() @ w[e].double().t() if op == "fwd" else dy[a:b].double() @ w[e].double()
            _same(got[a:b], ref, "rows of expert %d" % e)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,group", t.FORMATS)
@pytest.mark.parametrize("N,K", [(2048, 7168), (576, 18432), (7168, 2048)])
def test_one_block_of_k_a_row(m, dtype, fmt, group, N, K):
    # each row of x holds one block of 32 k, so a result is that block's sum: every run, stage and window of scales,
    # their ends and the last k among them
    q, s = _weights4((N, K), group, fmt, N)
    w = _values(q, s, group).t()
    for M in (1, 16, 31, 64):
        print("one block", dtype, fmt, group, M, N, K, flush=True)
        for first in range(0, K // 32, M) if M > 16 else (0, 31, K // 64 - 1, K // 64, K // 32 - 1):
            blocks = (first + torch.arange(M, device=DEV)) % (K // 32)
            keep = torch.arange(K, device=DEV)[None] // 32 == blocks[:, None]
            x = torch.where(keep, _whole((M, K), dtype, first), 0)
            _same(m.gemm_fp4_groupscale(x, q, s, group), x.double() @ w, "%d rows from block %d" % (M, first))


def _rms(v):
    return float(v.square().mean().sqrt())


def _long_sum(got, ref, K, dtype, what):
    half = torch.exp2(torch.floor(torch.log2(ref.abs())) - (8 if dtype == "bf16" else 11))
    bound = 1.1 * _rms(half) / 3 ** 0.5 + (K / 32 + 8) * 2.0 ** -23 * _rms(ref)
    err = _rms(got.double() - ref)
    assert err <= bound, "%s: RMS error %.3g above %.3g" % (what, err, bound)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt,group", t.FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 18432, 7168), (16, 2048, 7168), (20, 2048, 7168), (64, 2048, 7168), (64, 576, 18432),
                                   (48, 7168, 2048)])
def test_long_sums(m, dtype, fmt, group, M, N, K):
    print("long sum", dtype, fmt, group, M, N, K, flush=True)
    x = torch.randn((M, K), generator=_gen(M), device=DEV).to(DT[dtype])
    w = (torch.randn((N, K), generator=_gen(N), device=DEV) * 0.02).to(DT[dtype])
    q, s = m.fp4_quant_groups(w, group, fmt)
    ref = x.double() @ _values(q, s, group).t()
    _long_sum(m.gemm_fp4_groupscale(x, q, s, group), ref, K, dtype, "linear")
    off = torch.tensor([0, M // 2, M // 2, M], dtype=torch.int32, device=DEV)
    c = m.grouped_gemm_fp4(x, q.expand(3, -1, -1).contiguous(), s.expand(3, -1, -1).contiguous(), off, group)
    _long_sum(c, ref, K, dtype, "experts")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,N,K", [(40, 2048, 7168), (600, 1000, 7168)])
def test_long_sums_of_ragged_products(m, dtype, R, N, K):
    print("long sum, ragged", dtype, R, N, K, flush=True)
    off = torch.tensor([0, R // 3, R // 3, R - 7, R, R, R, R], dtype=torch.int32, device=DEV)
    x, dy = (torch.randn((R, c), generator=_gen(c), device=DEV).to(DT[dtype]) for c in (K, N))
    w = (torch.randn((7, N, K), generator=_gen(R), device=DEV) * 0.02).to(DT[dtype])
    o = off.tolist()
    seg = [(e, o[e], o[e + 1]) for e in range(7)]
    ref = torch.cat([x[a:b].double() @ w[e].double().t() for e, a, b in seg])
    _long_sum(m.grouped_gemm(x, w, off), ref, K, dtype, "y")
    ref = torch.cat([dy[a:b].double() @ w[e].double() for e, a, b in seg])
    _long_sum(m.grouped_gemm_dgrad(dy, w, off), ref, N, dtype, "dx")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("spread", [12, 13, 14, 22])
@pytest.mark.parametrize("N,K,rows", [(40, 512, (1, 7, 16, 24, 64)), (40, 7168, (1, 16, 40)), (600, 2048, (12, 64)), (33000, 256, (2, 8, 20, 64))])
def test_scales_far_apart_in_whole_dwords(m, dtype, spread, N, K, rows):
    # groups of 32 whose scale rows are whole dwords; neighbours' powers of two up to 2^spread apart in some columns, x
    # in one group in some rows, so that the smallest scales' products are whole results
    rng = np.random.default_rng(spread)
    q, s = rng.integers(0, 256, (N, K // 2), dtype=np.uint8), np.full((N, K // 32), 121, np.uint8)
    s[::3] = 125 - rng.choice([0, spread // 2, spread], s[::3].shape).astype(np.uint8)
    w = fp4.dequant_groups(q, s, 32)
    qd, sd = torch.tensor(q, device=DEV), torch.tensor(s, device=DEV)
    for M in rows:
        print("scales apart", dtype, spread, M, N, K, flush=True)
        x = (torch.randn((M, K), generator=torch.Generator().manual_seed(M)) * 8).to(DT[dtype])
        for r in range(1, M, 2):
            lo = r // 2 % (K // 32) * 32
            x[r, :lo], x[r, lo + 32:] = 0, 0
        xf = x.double().numpy()
        ref, d = xf @ w.T, (K + 8) * 2.0 ** -23 * (np.abs(xf) @ np.abs(w).T)
        lo, hi = (torch.tensor(v).to(DT[dtype]).double().numpy() for v in (ref - d, ref + d))
        one = m.gemm_fp4_groupscale(x.to(DEV), qd, sd, 32)
        both = m.grouped_gemm_fp4(x.to(DEV), qd[None], sd[None], torch.tensor([0, M], dtype=torch.int32, device=DEV), 32)
        for got in (one.double().cpu().numpy(), both.double().cpu().numpy()):
            assert ((got >= lo) & (got <= hi)).all(), (M, N, K)


@pytest.mark.parametrize("fmt", ["fp32", "e8m0"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_pack_subnormal_weights(m, fmt, group):
    # groups whose largest value is a subnormal bf16, down to the smallest one
    rng = np.random.default_rng(group)
    w = torch.tensor(rng.normal(size=(64, 256)) * np.ldexp(1.0, -np.arange(124, 140).repeat(4))[:, None]).to(torch.bfloat16)
    assert bool((w.float().abs()[8:] < 2.0 ** -126).any()) and bool((w != 0).any(1)[:32].all())
    q, s = m.fp4_quant_groups(w.to(DEV), group, fmt)
    rq, rs = fp4.quant_groups(w.float().numpy(), group, fmt == "e8m0")
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)
    ref = torch.tensor(fp4.dequant_groups(rq, rs, group).astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(m.fp4_dequant_groups(q, s, group).cpu().view(torch.int16), ref.view(torch.int16))
