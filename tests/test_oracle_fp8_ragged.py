"""Pins of the FP8 operands' oracle: the scale's definition by search, torch's float8 cast, and the blocks' numbering."""
import numpy as np
import pytest
import torch

from oracle import fp8, fp8_ragged as o


def test_scale_is_the_smallest_power_that_fits():
    for amax in [448.0, 449.0, 447.0, 896.0, 1.0, 1.75, 1.7500001, 1.7499999, 3.0e38, 2.0 ** -126, 2.0 ** -133, 2.0 ** -119, 0.875]:
        c = int(o.e8m0_byte(amax))
        s = 2.0 ** (c - 127)
        assert amax / s <= 448 and (c == 0 or amax / (s / 2) > 448), amax
    assert o.e8m0_byte(0.0) == 127 and o.e8m0_byte(np.inf) == 255 and o.e8m0_byte(np.nan) == 255


@pytest.mark.parametrize("rows", [1, 128])
def test_codes_are_torchs(rows):
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn((130, 200), generator=g) * torch.logspace(-20, 15, 200)).to(torch.bfloat16)
    x[0] = 0
    q, s = o.quant_blocks(x.double().numpy(), rows)
    each = np.repeat(np.repeat(o.e8m0_value(s), rows, 0)[:130], 128, 1)[:, :200]
    ref = (x.double() / torch.tensor(each)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (q == ref).all()
    v = o.values(q, s, rows)
    err = np.abs(v - x.double().numpy())
    # half a step of 3 mantissa bits, or half of the smallest step
    assert (err <= np.maximum(np.abs(v) / 15, each * 2.0 ** -10)).all()


def test_fp32_scales_are_those_of_the_activation_quantiser():
    from oracle import quant
    g = torch.Generator().manual_seed(5)
    x = torch.randn((4, 300), generator=g).to(torch.bfloat16).float().numpy()
    q, s = o.quant_blocks(x, 1, "fp32")
    rq, rs = quant.quant_1x128(x)
    assert (q == rq).all() and (s == rs).all()


def test_column_blocks_never_meet_and_hold_the_rows():
    g = np.random.default_rng(7)
    for _ in range(200):
        E = int(g.integers(1, 9))
        counts = g.integers(0, 300, E) * g.integers(0, 2, E)
        lead, tail = int(g.integers(0, 200)), int(g.integers(0, 200))
        offsets = (lead + np.concatenate([[0], np.cumsum(counts)])).tolist()
        R = offsets[-1] + tail
        x = g.normal(size=(R, 2))
        qt, s, used = o.quant_columns(x, offsets)      # asserts that no two segments share a block
        assert used.sum() == sum(-(-c // 128) for c in counts)
        e = int(g.integers(0, E))
        v = o.column_values(qt, s, offsets, e)
        rows = x[offsets[e]:offsets[e + 1]]
        assert (v[len(rows):] == 0).all()
        assert (np.abs(v[:len(rows)] - rows) <= np.abs(rows) / 15 + 2.0 ** -10 * np.abs(rows).max(initial=0)).all()


def test_wgrad_of_exact_codes_is_the_product():
    g = np.random.default_rng(8)
    offsets = [0, 5, 5, 150]
    # whole numbers up to 8 are e4m3 values at any power-of-two scale that keeps them whole or better
    dy, x = g.integers(-8, 9, (150, 3)).astype(float), g.integers(-8, 9, (150, 4)).astype(float)
    dw, mag = o.wgrad(*o.quant_columns(dy, offsets)[:2], *o.quant_columns(x, offsets)[:2], offsets)
    for e in range(3):
        a, b = offsets[e], offsets[e + 1]
        assert (dw[e] == dy[a:b].T @ x[a:b]).all() and (mag[e] == np.abs(dy[a:b]).T @ np.abs(x[a:b])).all()
    assert fp8.decode(fp8.encode(np.float32(8))) == 8


def test_unit_sum_lies_within_its_bound():
    g = np.random.default_rng(9)
    qa, qb = g.integers(0, 256, (20, 64)).astype(np.uint8), g.integers(0, 256, (24, 64)).astype(np.uint8)
    for q in (qa, qb):
        q[(q & 127) == 127] = 0
        q[:, :16] &= 0x8f                         # zeros and subnormal codes
    sa, sb = np.ones(qa.shape), np.full(qb.shape, 0.25)
    exact = (fp8.decode(qa) * sa) @ (fp8.decode(qb) * sb).T
    got, d = o.unit_sum(qa, sa, qb, sb), o.unit_bound(qa, sa, qb, sb)
    assert (np.abs(got - exact) <= d * (1 + 1e-12) + 1e-12 * np.abs(exact).max()).all() and (got != exact).any()
    # products within 2^-7 of the largest lose nothing
    qa, qb = g.integers(0x38, 0x40, (4, 64)).astype(np.uint8), g.integers(0x38, 0x48, (5, 64)).astype(np.uint8)
    one = np.ones((5, 64))
    assert (o.unit_sum(qa, one[:4], qb, one) == fp8.decode(qa) @ fp8.decode(qb).T).all()
