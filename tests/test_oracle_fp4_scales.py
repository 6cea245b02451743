"""Pins of the 4-bit oracle's scales (CPU only): where a group's largest value lands."""
import numpy as np
import pytest

from oracle import fp4


@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_the_largest_of_a_group(rng, e8m0, group):
    w = rng.normal(0, 0.02, (9, 224)).astype(np.float32)
    q, s = fp4.quant_groups(w, group, e8m0)
    v, sv = fp4.dequant_groups(q, s, group), fp4.scale_values(s)
    for g in range(-(-224 // group)):
        part, back = w[:, g * group:(g + 1) * group], v[:, g * group:(g + 1) * group]
        at = np.abs(part).argmax(-1)[:, None]
        top, got = np.take_along_axis(part, at, -1)[:, 0].astype(np.float64), np.take_along_axis(back, at, -1)[:, 0]
        if e8m0:    # s is the power of two with 4 s <= amax < 8 s; 6 s from the tie at 5 s on
            assert (4 * sv[:, g] <= np.abs(top)).all() and (np.abs(top) < 8 * sv[:, g]).all()
            assert np.array_equal(got, np.sign(top) * np.where(np.abs(top) > 5 * sv[:, g], 6, 4) * sv[:, g])
        else:       # the code of 6 over s = amax / 6
            assert np.array_equal(got, np.sign(top) * 6 * sv[:, g])
            assert (np.abs(got - top) <= 2.0 ** -23 * np.abs(top)).all()
        assert (np.abs(back) <= np.abs(got)[:, None]).all()


def test_weights_near_zero_and_saturated_ones():
    # what 4 bits may lose of a value: all of it below s / 4, a quarter of it at the top of an E8M0 group
    w = np.zeros((1, 32), np.float32)
    w[0, :3] = 7.999, 0.2499, 0.2501
    q, s = fp4.quant_groups(w, 32, True)
    assert s[0, 0] == 127 and np.array_equal(fp4.dequant_groups(q, s, 32)[0, :3], [6.0, 0.0, 0.5])
