"""Pins of the dispatch oracle: torch's stable sort, a permutation matrix, differences."""
import numpy as np
import pytest
import torch

from oracle import dispatch


def _ids(T, k, E, seed, outside):
    g = np.random.default_rng(seed)
    return g.integers(-2 if outside else 0, E + (3 if outside else 0), (T, k))


@pytest.mark.parametrize("T,k,E,outside", [(1, 1, 1, False), (7, 3, 5, False), (40, 8, 9, True), (16, 4, 64, True), (0, 2, 3, False)])
def test_group_is_the_stable_order(T, k, E, outside):
    ids = _ids(T, k, E, T + k, outside)
    off, rop, por = dispatch.group(ids, E)
    flat = torch.tensor(ids.reshape(-1))
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices.numpy()
    n = int((key < E).sum())
    assert off[0] == 0 and off[-1] == n and (np.diff(off) == np.bincount(key[key < E].numpy(), minlength=E)).all()
    assert (por[:n] == order[:n]).all() and (por[n:] == -1).all()
    assert (rop.reshape(-1)[por[:n]] == np.arange(n)).all() and ((rop >= 0) == (key < E).numpy().reshape(T, k)).all()


def test_combine_is_a_matrix_and_its_gradients_its_transpose():
    g = np.random.default_rng(3)
    T, k, E, H = 9, 3, 5, 6
    off, rop, _ = dispatch.group(_ids(T, k, E, 4, True), E)
    w, rows, dout, x = g.normal(size=(T, k)), g.normal(size=(T * k, H)), g.normal(size=(T, H)), g.normal(size=(T, H))
    P = np.zeros((T, T * k))
    for (t, j), r in np.ndenumerate(rop):
        if r >= 0:
            P[t, r] = w[t, j]
    out, mag = dispatch.combine(rows, rop, w)
    np.testing.assert_allclose(out, P @ rows, atol=1e-12)
    np.testing.assert_allclose(mag, np.abs(P) @ np.abs(rows), atol=1e-12)
    kept = g.normal(size=rows.shape)
    drows, dw, _ = dispatch.combine_grad(dout, rows, rop, w, kept)
    has = np.abs(P).sum(0) > 0
    np.testing.assert_allclose(drows[has], (P.T @ dout)[has], atol=1e-12)
    assert (drows[~has] == kept[~has]).all()
    # the sum is linear in the weights: a difference of any size is the derivative
    for t, j in ((0, 0), (3, 2), (8, 1)):
        step = np.zeros_like(w)
        step[t, j] = 1.0
        up = (dispatch.combine(rows, rop, w + step)[0] * dout).sum() - (out * dout).sum()
        assert abs(up - dw[t, j]) < 1e-10
    rows0 = dispatch.dispatch(x, rop, np.zeros((T * k, H)))
    np.testing.assert_allclose(rows0, (P != 0).T @ x, atol=1e-12)
