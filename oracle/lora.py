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


def cancelling(seed, rows, K, N, R, n):
    """Integer data whose adapter sums base takes back but for a small rest.

    Every entry of x A^T is an integer of 18 to 20 bits (16 products of two
    integers of 8 bits), so a bf16 or fp16 rounding of it, or a bf16 one of
    what the first left over, shows in the rest. A column of B has at most 8
    entries, all 1 or -1: every partial sum stays below 2^24, exact in fp32.
    Returns x, a, b, ids, base, rest as float64 / int64; out equals rest,
    integers up to 100, exact in every type."""
    rng = np.random.default_rng(seed)
    used = min(16, K)
    x = np.zeros((rows, K))
    for t in range(rows):
        x[t, rng.choice(K, used, replace=False)] = rng.integers(128, 256, used)
    a = rng.integers(128, 256, (n, R, K)).astype(np.float64)
    b = np.zeros((n, N, R))
    for i in range(n):
        for c in range(N):
            at = rng.choice(R, min(8, R), replace=False)
            b[i, c, at] = rng.integers(0, 2, at.size) * 2 - 1
    ids = rng.integers(-1, n, rows)
    rest = rng.integers(-100, 101, (rows, N)).astype(np.float64)
    base = rest - lora(x, a, b, ids)
    return x, a, b, ids, base, rest
