"""Rows carried to experts and back (oracle side), in float64, one choice at a
time. pos [rows, topk]: packed position of each choice, outside [0, rows * topk)
where it takes no part. The definitions are this library's own."""

import numpy as np


def _choices(pos):
    pos = np.asarray(pos)
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            if 0 <= pos[t, j] < pos.size:
                yield t, j, pos[t, j]


def permute(x, pos, out):
    """out (a copy of it) with x[t] at every choice's position."""
    out = np.array(out, dtype=np.float64)
    for t, _, q in _choices(pos):
        out[q] = x[t]
    return out


def unpermute(y, pos, w=None):
    out = np.zeros((np.asarray(pos).shape[0], y.shape[1]))
    for t, j, q in _choices(pos):
        out[t] += (1.0 if w is None else w[t, j]) * y[q]
    return out


def unpermute_backward(dout, y, pos, w, dy):
    """(dy, dw); dy starts as a copy of the one given."""
    dy = np.array(dy, dtype=np.float64)
    dw = np.zeros(np.asarray(pos).shape)
    for t, j, q in _choices(pos):
        dy[q] = (1.0 if w is None else w[t, j]) * dout[t]
        if y is not None:
            dw[t, j] = np.dot(dout[t], y[q])
    return dy, dw
