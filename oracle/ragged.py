"""Products grouped by expert over ragged row segments, in numpy binary64.

Expert e owns rows [offsets[e], offsets[e+1]).  Each function also returns the sums of the
absolute products, which bound the rounding of any order of summation.
"""
import numpy as np


def forward(x, w, offsets):
    """y[r] = w[e(r)] x[r]; rows in no segment are NaN.  (y, sum of |x||w|)"""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    mag = np.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = x[a:b] @ w[e].T
        mag[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, mag


def dgrad(dy, w, offsets):
    return forward(dy, np.swapaxes(np.asarray(w, np.float64), 1, 2), offsets)


def wgrad(dy, x, offsets):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    E = len(offsets) - 1
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    mag = np.zeros_like(dw)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        dw[e] = dy[a:b].T @ x[a:b]
        mag[e] = np.abs(dy[a:b]).T @ np.abs(x[a:b])
    return dw, mag
