"""Tokens to the rows of their experts and back, in numpy (binary64 where there is arithmetic)."""
import numpy as np


def group(topk_ids, E):
    """(offsets [E+1], row_of_pair [T, k], pair_of_row [T*k]): pairs by expert, ascending inside an expert; -1 for
    pairs whose id is outside [0, E) and for the rows behind the last segment."""
    ids = np.asarray(topk_ids)
    T, k = ids.shape
    offsets = np.zeros(E + 1, np.int64)
    pair_of_row = []
    for e in range(E):
        pair_of_row += [p for p, i in enumerate(ids.reshape(-1).tolist()) if i == e]
        offsets[e + 1] = len(pair_of_row)
    row_of_pair = np.full(T * k, -1, np.int64)
    row_of_pair[pair_of_row] = np.arange(len(pair_of_row))
    return offsets, row_of_pair.reshape(T, k), np.array(pair_of_row + [-1] * (T * k - len(pair_of_row)), np.int64)


def dispatch(x, row_of_pair, rows):
    """`rows` with x[t] in the rows of token t's pairs."""
    out = np.array(rows)
    for (t, j), r in np.ndenumerate(row_of_pair):
        if 0 <= r < out.shape[0]:
            out[r] = x[t]
    return out


def combine(rows, row_of_pair, weights=None):
    """(out, sum of |weight||row|): out[t] = sum_j weights[t, j] rows[row_of_pair[t, j]]."""
    rows = np.asarray(rows, np.float64)
    out = np.zeros((row_of_pair.shape[0], rows.shape[1]))
    mag = np.zeros_like(out)
    for (t, j), r in np.ndenumerate(row_of_pair):
        if 0 <= r < rows.shape[0]:
            w = 1.0 if weights is None else float(weights[t, j])
            out[t] += w * rows[r]
            mag[t] += np.abs(w * rows[r])
    return out, mag


def combine_grad(dout, rows, row_of_pair, weights, drows):
    """(drows, dweights, sum of |dout||row|) of combine; rows that no pair has stay as in the given drows."""
    dout, rows, drows = (np.array(a, np.float64) for a in (dout, rows, drows))
    dw, mag = np.zeros(row_of_pair.shape), np.zeros(row_of_pair.shape)
    for (t, j), r in np.ndenumerate(row_of_pair):
        if 0 <= r < rows.shape[0]:
            drows[r] = float(weights[t, j]) * dout[t]
            dw[t, j] = dout[t] @ rows[r]
            mag[t, j] = np.abs(dout[t]) @ np.abs(rows[r])
    return drows, dw, mag
