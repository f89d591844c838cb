"""Products with 4-bit weights and group scales (oracle side), in float64:
out[p, n] = sum_k x[p, k] scale[e, n, k // G] (q[e, n, k] - zero[e, n, k // G]).
The definition and the tile layout are this library's own."""

import numpy as np


def weights(q, scale, zero=None):
    """[experts, out, in] from q [experts, out, in / 2], two weights a byte."""
    q = np.asarray(q)
    E, N, half = q.shape
    v = np.empty((E, N, 2 * half))
    v[:, :, 0::2] = q & 15
    v[:, :, 1::2] = q >> 4
    G = 2 * half // scale.shape[2]
    z = 8.0 if zero is None else np.repeat(np.asarray(zero, np.float64), G, axis=2)
    return (v - z) * np.repeat(np.asarray(scale, np.float64), G, axis=2)


def linear(x, w, offset=None, out=None):
    """out (a copy of it, zeros by default) with the experts' rows filled."""
    x = np.asarray(x, np.float64)
    out = np.zeros((x.shape[0], w.shape[1])) if out is None else np.array(out, np.float64)
    offset = [0, x.shape[0]] if offset is None else offset
    for e in range(w.shape[0]):
        a, b = int(offset[e]), int(offset[e + 1])
        out[a:b] = x[a:b] @ w[e].T
    return out


# Where an input stands in its word: bits 4 p hold this one of eight.
ORDER = [0, 2, 4, 6, 1, 3, 5, 7]


def tile_word(v, nt, kt, lane, i):
    """Word i of a lane of tile (nt, kt) from an expert's values [out, in]."""
    n, kg = 16 * nt + lane % 16, lane // 16
    word = 0
    for p, j in enumerate(ORDER):
        k = 128 * kt + 32 * i + 8 * kg + j
        if n < v.shape[0] and k < v.shape[1]:
            word |= int(v[n, k]) << (4 * p)
    return word
