"""The 4-bit products and those grouped by expert.  TEST INFRASTRUCTURE (oracle).

Plain numpy in 64 bits over inputs already widened from their storage types, one
expert after another; formulas are those include/pe.h states.
"""
import numpy as np

from . import dense


def group_rows(ids, E):
    """(offsets [E + 1], rows, places [T, k]): entries by expert, -1 where the id is outside [0, E)."""
    T, k = ids.shape
    places = np.full((T, k), -1, np.int32)
    offsets, rows = [0], []
    for e in range(E):
        for t in range(T):
            for j in range(k):
                if ids[t, j] == e:
                    places[t, j] = len(rows)
                    rows.append(t)
        offsets.append(len(rows))
    return np.array(offsets, np.int32), np.array(rows, np.int32), places


def linear(x, w, bias, act_name, offsets, rows, R):
    """y [R, N], NaN in the rows behind the last expert's."""
    y = np.full((R, w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        p = np.arange(offsets[e], offsets[e + 1])
        xe = x[p if rows is None else rows[p]]
        y[p] = dense.linear(xe, w[e], None if bias is None else bias[e], act_name, None)
    return y


def combine(y, places, w, residual):
    T, k = places.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.astype(np.float64).copy()
    for t in range(T):
        for j in range(k):
            if 0 <= places[t, j] < y.shape[0]:
                out[t] += (1.0 if w is None else w[t, j]) * y[places[t, j]]
    return out


def combine_backward(dout, places, w, y):
    """(dy with NaN in rows that no place names, dw)."""
    T, k = places.shape
    dy, dw = np.full(y.shape, np.nan), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = places[t, j]
            if 0 <= p < y.shape[0]:
                dy[p] = (1.0 if w is None else w[t, j]) * dout[t]
                dw[t, j] = dout[t] @ y[p]
    return dy, dw
