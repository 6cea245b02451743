"""Pins of the 4-bit weight oracle and of the ragged product oracle (CPU only)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import fp4, ragged


def test_levels_follow_the_format():
    # e2m1: 1 sign, 2 exponent (bias 1), 1 mantissa bit; exponent field 0 is subnormal
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        v = m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        assert fp4.decode(c) == (-v if c & 8 else v)
    assert np.signbit(fp4.decode(8))


def test_encode_is_nearest_with_ties_to_even(rng):
    y = np.concatenate([rng.normal(0, 3, 4000), np.arange(-64, 65) / 8.0, [1e30, -1e30, 1e-30]])
    got = fp4.encode(y)
    for v, c in zip(y, got):
        d = np.abs(fp4.LEVELS - min(abs(v), 1e3))
        best = np.flatnonzero(d == d.min())
        want = best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]
        assert c & 7 == want and bool(c & 8) == bool(np.signbit(v)), v


def test_pack_round_trip(rng):
    c = rng.integers(0, 16, (5, 64)).astype(np.uint8)
    assert np.array_equal(fp4.unpack(fp4.pack(c)), c)
    assert fp4.pack(c)[0, 0] == c[0, 0] | (c[0, 1] << 4)


@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quant_properties(rng, e8m0, group):
    w = rng.normal(0, 0.02, (7, 224)).astype(np.float32)
    w[0] = 0
    w[1, :3] = [np.nan, np.inf, 1]
    q, s = fp4.quant_groups(w, group, e8m0)
    v = fp4.dequant_groups(q, s, group)
    assert np.all(v[0] == 0) and np.isnan(v[1, :group]).all()
    assert (s[0] == (127 if e8m0 else 1)).all()
    sv = np.repeat(fp4.scale_values(s), group, -1)[:, :224]
    err = np.abs(v - w)[2:]
    # half a step of the level's binade, and what saturation cuts off (E8M0 reaches up to 8 s)
    assert (err <= np.where(np.abs(w[2:]) <= 6 * sv[2:], 1.0, 2.0) * sv[2:] * (1 + 1e-6)).all()
    if not e8m0:
        g0 = np.abs(w[2:, :group])
        assert np.array_equal(np.abs(v[2:, :group]).argmax(-1), g0.argmax(-1)) or (np.abs(v[2:, :group]).max(-1) > 0).all()


def test_reciprocal_quotient_is_the_ieee_quotient():
    """fl32(w / s) from the correctly rounded reciprocal r = fl32(1 / s) by q = fl(w r),
    q' = fl(q + r fl(w - q s)): over every significand of a 16-bit amax and weight, at every distance of
    exponents where a code other than 0 can result."""
    f = np.float32

    def check(bits):
        n = 1 << bits
        amax = (1 + np.arange(n, dtype=np.float64) / n).astype(f)
        for w_exp in range(-6, 1):                       # |w| < amax / 64 is code 0 whatever the rounding
            w = (amax * f(2.0 ** w_exp))[:, None]
            s = (amax / f(6))[None, :]
            r = f(1) / s
            q = w * r
            rem = (w.astype(np.float64) - q.astype(np.float64) * s.astype(np.float64)).astype(f)   # exact in binary64
            got = (q.astype(np.float64) + rem.astype(np.float64) * r.astype(np.float64)).astype(f)
            assert np.array_equal(got, w / s), (bits, w_exp)

    check(7)
    check(10)


def test_ragged_forward_and_gradients_agree_with_autograd(rng):
    off = [0, 3, 3, 8, 8]
    x, w = rng.normal(size=(8, 5)), rng.normal(size=(4, 6, 5))
    dy = rng.normal(size=(8, 6))
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = torch.cat([tx[off[e]:off[e + 1]] @ tw[e].T for e in range(4)])
    y.backward(torch.tensor(dy))
    assert np.allclose(ragged.forward(x, w, off)[0], y.detach().numpy())
    assert np.allclose(ragged.dgrad(dy, w, off)[0], tx.grad.numpy())
    assert np.allclose(ragged.wgrad(dy, x, off)[0], tw.grad.numpy())
    assert np.isnan(ragged.forward(x, w, [0, 3, 3, 7, 7])[0][7]).all()


def test_oracle_modules_are_listed():
    assert oracle.fp4 is fp4 and oracle.ragged is ragged
