"""Products on 4-bit weights with E8M0 scales from the ends of their range, against the formula in 64 bits.

Columns hold scale bytes of one kind: the largest, the smallest, ordinary ones, both in turn, or a NaN; rows of x are
ordinary, large, small, subnormal, zero, or zero in every other group, so that results in the normal range come out of
every kind of column.  Tolerance: an fp32 sum of K products in any order is within d = (K + 8) 2^-23 of the sum of their
magnitudes, and the output is rounded once, so it lies between the rounded ends of [reference - d, reference + d].
Results whose terms leave [2^-100, 2^120] are not compared: fp32 sums may overflow or lose bits there.
"""
import numpy as np
import pytest
import torch

from oracle import fp4, ragged

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def m():
    import fp8_block_scaled_grouped_amd as mod
    mod.lib()
    return mod


def _scales(shape, rng):
    """E8M0 bytes [.., N, G]: the kind of a row by its index."""
    s = rng.integers(120, 131, shape)
    odd = np.arange(shape[-1]) % 2 == 1
    kind = np.arange(shape[-2]) % 6
    s[..., kind == 0, :] = rng.choice([253, 254], s[..., kind == 0, :].shape)
    s[..., kind == 1, :] = rng.choice([0, 1, 2], s[..., kind == 1, :].shape)
    s[..., kind == 3, :] = np.where(odd, rng.integers(250, 255, s[..., kind == 3, :].shape), s[..., kind == 3, :])
    s[..., kind == 4, :] = np.where(odd, s[..., kind == 4, :], rng.integers(0, 2, s[..., kind == 4, :].shape))
    s[..., kind == 5, shape[-1] // 2] = 255
    return s.astype(np.uint8)


def _rows(M, K, group, dtype, rng, first=0):
    kind = (np.arange(M) + first) % 6
    exps = (0, -95, 110, 0, 0, -131) if dtype == "bf16" else (0, -18, 6, 0, 0, -23)
    x = rng.normal(size=(M, K)) * np.ldexp(1.0, np.array(exps)[kind])[:, None]
    x[(kind[:, None] == 3) & (np.arange(K) // group % 2 == 1)[None, :]] = 0
    x[kind == 4] = 0
    return torch.tensor(x).to(DT[dtype])


def _check(got, ref, mag, K, dtype, what):
    g = got.float().cpu().numpy().astype(np.float64)
    nan = np.isnan(mag)
    assert np.isnan(g[nan]).all(), what + ": a NaN scale has to give NaN"
    with np.errstate(invalid="ignore"):
        live = ~nan & (mag < (2.0 ** 120 if dtype == "bf16" else 6e4))
        live &= (mag == 0) | (np.abs(ref) > 2.0 ** -100) if dtype == "bf16" else True
    assert (live.sum(0) > 0).sum() * 6 >= live.shape[1] and (live.sum(1) > 0).any()
    d = (K + 8) * 2.0 ** -23 * mag
    lo, hi = (torch.tensor(np.where(live, v, 0)).to(DT[dtype]).double().numpy() for v in (ref - d, ref + d))
    bad = live & ~((g >= lo) & (g <= hi))
    assert not bad.any(), "%s: %d of %d outside, first at %s: %r not in [%r, %r]" % (
        what, bad.sum(), live.sum(), np.argwhere(bad)[0], g[bad][0], lo[bad][0], hi[bad][0])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K,rows", [(60, 512, (1, 6, 16, 24, 64)), (66, 1056, (1, 12, 18, 40)), (33000, 256, (3, 8, 12, 30, 64))])
def test_linear(m, dtype, group, N, K, rows):
    rng = np.random.default_rng(K + group)
    q, s = rng.integers(0, 256, (N, K // 2), dtype=np.uint8), _scales((N, -(-K // group)), rng)
    w = fp4.dequant_groups(q, s, group)
    qd, sd = torch.tensor(q, device=DEV), torch.tensor(s, device=DEV)
    for M in rows:
        for first in range(6 if M == 1 else 1):
            print("e8m0 range", dtype, group, N, K, M, first, flush=True)
            x = _rows(M, K, group, dtype, rng, first)
            xf = x.double().numpy()
            _check(m.gemm_fp4_groupscale(x.to(DEV), qd, sd, group), xf @ w.T, np.abs(xf) @ np.abs(w).T, K, dtype,
                   "%d x %d x %d from row kind %d" % (M, N, K, first))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts", [[0, 6, 1, 12, 0], [6, 24, 0, 18], [70, 40, 0, 30]])
def test_experts(m, dtype, group, counts):
    N, K = 78, 512
    rng = np.random.default_rng(len(counts) + group)
    off = [0] + np.cumsum(counts).tolist()
    q, s = rng.integers(0, 256, (len(counts), N, K // 2), dtype=np.uint8), _scales((len(counts), N, K // group), rng)
    x = _rows(off[-1], K, group, dtype, rng)
    print("e8m0 range, experts", dtype, group, counts, flush=True)
    c = m.grouped_gemm_fp4(x.to(DEV), torch.tensor(q, device=DEV), torch.tensor(s, device=DEV),
                           torch.tensor(off, dtype=torch.int32, device=DEV), group)
    _check(c, *ragged.forward(x.double().numpy(), fp4.dequant_groups(q, s, group), off), K, dtype, "experts")
