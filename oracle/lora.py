"""Low-rank adapters beside a shared projection (oracle side), in float64:
out_t = base_t + scale_a (x_t A_a^T) B_a^T with a = ids[t], or base_t where
ids[t] names no adapter. One row at a time; the definition is this library's
own."""

import numpy as np


def lora(x, a, b, ids, scale=None, ranks=None, base=None):
    x, a, b = (np.asarray(v, dtype=np.float64) for v in (x, a, b))
    n, R, _ = a.shape
    out = np.zeros((x.shape[0], b.shape[1]))
    for t, i in enumerate(np.asarray(ids).reshape(-1)):
        if base is not None:
            out[t] = base[t]
        if 0 <= i < n:
            r = R if ranks is None else min(max(int(ranks[i]), 0), R)
            s = a[i][:r] @ x[t]
            if scale is not None:
                s = s * float(scale[i])
            out[t] += b[i][:, :r] @ s
    return out


def magnitude(x, a, b, ids, scale=None, ranks=None, base=None):
    """The same sums over absolute values: what rounding errors are relative
    to."""
    return lora(np.abs(x), np.abs(a), np.abs(b), ids,
                None if scale is None else np.abs(scale), ranks,
                None if base is None else np.abs(base))
