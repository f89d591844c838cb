"""GPU: rows carried to experts and back, the gradient of that, and products
with 4-bit weights against float64 oracles (MI355X only).

Tolerances. An output is off by at most half a step of its type (relative
eps / 2, absolute half the smallest subnormal) plus what fp32 arithmetic loses
before it, u = 2^-24 of the sum of absolute terms for each rounding of the
longest chain:
  unpermute   one fma for each choice
  backward    dy: one product. dw: an fma for every value a lane takes
              (8 ceil(features / (8 lanes)), lanes the power of two that holds
              features / 8, at most 256), 6 additions in a wave, 3 across waves
  w4          a matrix instruction's sums are taken as 32 additions that may
              each cut off (2 u): 2 in all for every input, and an fma a group
Where all terms and sums are whole numbers (times one power of two) that fit
the type, results are compared as bytes.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import permute as operm  # noqa: E402
from oracle import router as orouter  # noqa: E402
from oracle import w4 as ow4  # noqa: E402
from trellis_quantized_moe_amd import exl3  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
MARK = 777.0  # what untouched places hold


def _say(*a):
    print(*a, flush=True)


def _np(t):
    return t.detach().cpu().double().numpy()


def _bytes(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def _same(a, b):
    return torch.equal(_bytes(a), _bytes(b))


def _wide(t, pad, dtype, fill=float("nan")):
    """t as a column slice of a wider buffer of `dtype` filled with `fill`."""
    r, c = t.shape
    buf = torch.full((r, c + pad), fill, dtype=dtype, device=DEV)
    buf[:, :c] = t.to(DEV)
    return buf[:, :c]


def _within(got, ref, dt, rel, mag):
    """|got - ref| <= half a step + rel * mag, and the same non-finite values."""
    got, ref = np.asarray(got), np.asarray(ref)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
    half = torch.finfo(dt).eps / 2
    err = np.abs(got - ref)[fin]
    tol = (np.abs(ref) * half + TINY[dt] + rel * mag * (1 + half))[fin]
    assert np.all(err <= tol), "max excess %.3g" % np.max(err / np.maximum(tol, 1e-300))


def _meta(T, k, E, seed, dropped=0.2):
    g = torch.Generator().manual_seed(seed)
    ids = torch.argsort(torch.rand(T, E, generator=g), dim=1)[:, :k].to(torch.int32)
    ids[torch.rand(T, k, generator=g) < dropped] = -1
    return exl3.exl3_route_pack(ids.contiguous().to(DEV), torch.ones(T, k, device=DEV), E)


def _pos(meta, T, k):
    return meta["pos_of_pair"].cpu().numpy().reshape(T, k)


# ----------------------------------------------------------- rows to experts
MOVES = [(1, 1, 8), (1, 8, 64), (3, 2, 1024), (5, 32, 8), (17, 3, 520), (33, 8, 2048),
         (64, 9, 1032), (130, 4, 4104), (9, 16, 65536), (1000, 5, 264)]


@pytest.mark.parametrize("T,k,H", MOVES)
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_permute(T, k, H, dt):
    _say("permute", T, k, H, dt)
    meta = _meta(T, k, 40, T + k)
    g = torch.Generator().manual_seed(H)
    x = _wide(torch.randn(T, H, generator=g), 8, DT[dt])
    x[0, 0] = float("nan")
    out = torch.full((T * k, H + 16), MARK, dtype=DT[dt], device=DEV)
    exl3.exl3_permute(x, meta, k, out=out[:, 8:8 + H])
    want = torch.full_like(out, MARK)
    for t, j in np.argwhere(_pos(meta, T, k) >= 0):
        want[int(_pos(meta, T, k)[t, j]), 8:8 + H] = x[t]
    assert _same(out, want)


@pytest.mark.parametrize("T,k,H", MOVES)
@pytest.mark.parametrize("y_dt,w_dt,o_dt,pad", [
    ("f16", "f32", "f16", 0), ("bf16", "bf16", "f32", 8), ("f32", "f16", "bf16", 0),
    ("f32", None, "f32", 8), ("bf16", "f32", "f16", 0), ("f16", "f16", "bf16", 16),
    ("f16", None, "f32", 0), ("bf16", "f16", "bf16", 0), ("f32", "bf16", "f16", 0)])
def test_unpermute(T, k, H, y_dt, w_dt, o_dt, pad):
    _say("unpermute", T, k, H, y_dt, w_dt, o_dt)
    meta = _meta(T, k, 40, T + k)
    g = torch.Generator().manual_seed(H)
    y = _wide(torch.randn(T * k, H, generator=g), pad, DT[y_dt])
    kept = int(meta["expert_offset"][-1])
    y[kept:] = float("nan")  # not read
    w = None if w_dt is None else torch.randn(T, k, generator=g).to(DT[w_dt]).to(DEV)
    out = torch.full((T, H + pad), MARK, dtype=DT[o_dt], device=DEV)
    exl3.exl3_unpermute(y, meta, k, w, out=out[:, :H])
    pos, yn, wn = _pos(meta, T, k), _np(y), None if w is None else _np(w)
    yn[kept:] = 0
    ref = operm.unpermute(yn, pos, wn)
    mag = operm.unpermute(np.abs(yn), pos, None if w is None else np.abs(wn))
    _within(_np(out[:, :H]), ref, DT[o_dt], k * U, mag)
    assert (out[:, H:] == MARK).all()
    alone = exl3.exl3_unpermute(y, meta, k, w, out_dtype=DT[o_dt])
    assert _same(alone, out[:, :H])


@pytest.mark.parametrize("T,k,H", MOVES)
@pytest.mark.parametrize("y_dt,w_dt,o_dt,pad", [
    ("f16", "f32", "f16", 0), ("bf16", "bf16", "f32", 8), ("f32", "f16", "bf16", 0),
    ("f32", None, "f32", 8), ("bf16", "f32", "f16", 0), ("f16", "f16", "bf16", 16),
    ("f16", None, "f32", 0), ("bf16", "f16", "bf16", 0), ("f32", "bf16", "f16", 0)])
def test_unpermute_backward(T, k, H, y_dt, w_dt, o_dt, pad):
    _say("backward", T, k, H, y_dt, w_dt, o_dt)
    meta = _meta(T, k, 40, T + k)
    g = torch.Generator().manual_seed(H + 1)
    y = _wide(torch.randn(T * k, H, generator=g), pad, DT[y_dt])
    kept = int(meta["expert_offset"][-1])
    y[kept:] = float("nan")
    w = None if w_dt is None else torch.randn(T, k, generator=g).to(DT[w_dt]).to(DEV)
    dout = _wide(torch.randn(T, H, generator=g), pad, DT[o_dt])
    dy = torch.full((T * k, H + pad), MARK, dtype=DT[y_dt], device=DEV)
    got, dw = exl3.exl3_unpermute_backward(dout, meta, k, y, w, dy=dy[:, :H])
    pos, yn, dn = _pos(meta, T, k), _np(y), _np(dout)
    yn[kept:] = 0
    wn = None if w is None else _np(w)
    rdy, rdw = operm.unpermute_backward(dn, yn, pos, wn, np.full((T * k, H), MARK))
    assert got.data_ptr() == dy.data_ptr() and (dy[:, H:] == MARK).all()
    assert (dy[kept:] == MARK).all()
    assert dw.dtype == (DT[w_dt] if w_dt else torch.float32)
    _within(_np(got), rdy, DT[y_dt], U if y_dt != "f32" else 0, np.abs(rdy))
    lanes = 1
    while lanes < H // 8 and lanes < 256:
        lanes *= 2
    chain = 8 * -(-H // (8 * lanes)) + 9
    _, mag = operm.unpermute_backward(np.abs(dn), np.abs(yn), pos, wn, np.zeros((T * k, H)))
    _within(_np(dw), rdw, dw.dtype, chain * U, mag)
    only, none = exl3.exl3_unpermute_backward(dout, meta, k, w=w, dy_dtype=DT[y_dt])
    assert none is None and _same(only[:kept], got[:kept])


@pytest.mark.parametrize("dt,w_dt", [("f16", "f32"), ("bf16", "bf16"), ("f32", None)])
def test_moves_of_more_than_the_l2s_hold(dt, w_dt):
    """Large results take other stores: the rows of small calls, byte for byte."""
    T, k, H = 9000, 3, 2056
    meta = _meta(T, k, 11, 4)
    pos = meta["pos_of_pair"].view(T, k)
    kept = int(meta["expert_offset"][-1])
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, H, generator=g, device=DEV).to(DT[dt])
    w = None if w_dt is None else torch.rand(T, k, generator=g, device=DEV).to(DT[w_dt])
    zeros = torch.zeros(T * k, H, dtype=DT[dt], device=DEV)
    xs = exl3.exl3_permute(x, meta, k, out=zeros.clone())
    out = exl3.exl3_unpermute(xs, meta, k, w)
    dy, dw = exl3.exl3_unpermute_backward(x, meta, k, xs, w, dy=zeros.clone())
    want = zeros.clone()
    flat = pos.reshape(-1).long()
    held = flat >= 0
    want[flat[held]] = x.repeat_interleave(k, 0)[held]
    assert _same(xs, want) and (xs[kept:] == 0).all() and (dy[kept:] == 0).all()
    for lo in (0, 4321, T - 20):  # 20 rows, their packed rows moved to the front
        p = pos[lo:lo + 20].reshape(-1).long()
        part = torch.full((20 * k,), -1, dtype=torch.int32, device=DEV)
        part[p >= 0] = torch.arange(int((p >= 0).sum()), dtype=torch.int32, device=DEV)
        few = {"pos_of_pair": part}
        rows = p[p >= 0]
        y = zeros[:20 * k].clone()
        y[:rows.numel()] = xs[rows]
        pw = None if w is None else w[lo:lo + 20].contiguous()
        assert _same(exl3.exl3_unpermute(y, few, k, pw), out[lo:lo + 20])
        sy, sw = exl3.exl3_unpermute_backward(x[lo:lo + 20], few, k, y, pw)
        assert _same(sy[:rows.numel()], dy[rows]) and _same(sw, dw[lo:lo + 20])


def test_gradients_against_differences():
    """Whole numbers: every value and difference is exact, so the directional
    derivative along each single input equals the gradient's entry."""
    T, k, H, E = 6, 3, 16, 5
    meta = _meta(T, k, E, 3)
    kept = int(meta["expert_offset"][-1])
    g = torch.Generator().manual_seed(0)

    def ints(*s):
        return torch.randint(-4, 5, s, generator=g).float().to(DEV)

    x, y, w, dout = ints(T, H), ints(T * k, H), ints(T, k), ints(T, H)
    dxs = ints(T * k, H)
    dy, dw = exl3.exl3_unpermute_backward(dout, meta, k, y, w)
    dx = exl3.exl3_unpermute(dxs, meta, k)

    def back(y, w):
        return float((exl3.exl3_unpermute(y, meta, k, w) * dout).double().sum())

    def there(x):
        out = torch.zeros(T * k, H, device=DEV)
        return float((exl3.exl3_permute(x, meta, k, out=out) * dxs).double().sum())

    for a, f, grad in ((y, lambda a: back(a, w), dy), (w, lambda a: back(y, a), dw),
                       (x, there, dx)):
        for i in range(0, a.numel(), 7 if a.numel() > 20 else 1):
            if a is y and i // H >= kept:
                continue
            hi, lo = a.clone(), a.clone()
            hi.view(-1)[i] += 1
            lo.view(-1)[i] -= 1
            assert (f(hi) - f(lo)) / 2 == float(grad.reshape(-1)[i])


def test_rows_without_choices_and_strange_positions():
    """All choices dropped: zeros out, nothing carried, dw 0. Positions outside
    the packed rows take no part."""
    T, k, H = 5, 3, 64
    x = torch.randn(T, H, device=DEV)
    y = torch.full((T * k, H), float("nan"), device=DEV)
    for bad in (-1, T * k, 2 ** 31 - 1, -2 ** 31):
        meta = {"pos_of_pair": torch.full((T * k,), bad, dtype=torch.int32, device=DEV)}
        out = torch.full((T * k, H), MARK, device=DEV)
        assert (exl3.exl3_permute(x, meta, k, out=out) == MARK).all()
        assert not exl3.exl3_unpermute(y, meta, k).any()
        dy, dw = exl3.exl3_unpermute_backward(x, meta, k, y, dy=out)
        assert (dy == MARK).all() and not dw.any()


def test_special_values_stay_in_their_rows():
    inf, nan = float("inf"), float("nan")
    T, k, H = 40, 4, 128
    meta = _meta(T, k, 12, 9, dropped=0)
    y = torch.randn(T * k, H, device=DEV)
    w = torch.rand(T, k, device=DEV)
    clean = exl3.exl3_unpermute(y, meta, k, w)
    pos = _pos(meta, T, k)
    y[int(pos[3, 1])], y[int(pos[7, 0])] = nan, inf
    w[9, 2], w[11, 3] = 0.0, -inf
    y[int(pos[9, 2])] = inf  # 0 * inf
    got = exl3.exl3_unpermute(y, meta, k, w)
    rest = [t for t in range(T) if t not in (3, 7, 9, 11)]
    assert _same(got[rest], clean[rest])
    assert got[3].isnan().all() and (got[7] == inf).all() and got[9].isnan().all()
    assert not got[11].isfinite().any()
    dout = torch.randn(T, H, device=DEV)
    dout[5] = inf
    dy, dw = exl3.exl3_unpermute_backward(dout, meta, k, y, w)
    assert dw[3, 1].isnan() and not dw[7, 0].isfinite()
    assert (~dw[5].isfinite()).all() and dw[3, 0].isfinite() and dw[8].isfinite().all()
    assert dy[torch.tensor(pos[5], device=DEV).long()].isinf().all()


def test_moves_at_a_large_distance():
    """Element offsets past 2^32: rows 2^19 elements apart."""
    T, k, H, ld = 9001, 1, 16, 1 << 19
    meta = _meta(T, k, 7, 2, dropped=0.1)
    kept = int(meta["expert_offset"][-1])

    def far(t):
        buf = torch.empty(t.shape[0], ld, dtype=t.dtype, device=DEV)
        buf[:, :H] = t
        return buf[:, :H]

    x = torch.randn(T, H, device=DEV).half()
    xs = exl3.exl3_permute(x, meta, k, out=torch.zeros(T * k, H, device=DEV).half())
    fxs = exl3.exl3_permute(far(x), meta, k, out=far(torch.zeros(T * k, H, device=DEV).half()))
    assert _same(fxs, xs)
    w = torch.rand(T, k, device=DEV)
    out = exl3.exl3_unpermute(xs, meta, k, w)
    assert _same(exl3.exl3_unpermute(fxs, meta, k, w, out=far(out)), out)
    dy, dw = exl3.exl3_unpermute_backward(out, meta, k, xs, w)
    fdy, fdw = exl3.exl3_unpermute_backward(far(out), meta, k, fxs, w, dy=far(xs))
    assert _same(fdy[:kept], dy[:kept]) and _same(fdw, dw)


# ------------------------------------------------------------ 4-bit products
def _offsets(kind, rows, E, g):
    """expert_offset of `rows` packed rows."""
    if kind is None:
        return None
    if kind == "one":  # one row for each of the first experts, the rest empty
        o = torch.arange(E + 1).clamp(max=rows)
    elif kind == "last":  # empty experts before the only one in use
        o = torch.zeros(E + 1, dtype=torch.int64)
        o[E] = rows
    else:  # ragged, the last rows nobody's
        o = torch.randint(0, rows + 1, (E + 1,), generator=g).sort().values
        o[0] = 0
    return o.to(torch.int32)


W4 = [
    # rows, offsets, E, K, N, G, zeros, x, scale, out, pad
    (1, None, 1, 32, 8, 32, True, "f16", "f16", "f16", 0),
    (1, None, 1, 4096, 192, 128, False, "bf16", "bf16", "f32", 0),
    (2, None, 1, 96, 24, 32, False, "bf16", "f16", "bf16", 8),
    (15, None, 1, 1088, 40, 64, True, "f16", "bf16", "f32", 0),
    (16, None, 1, 640, 136, 128, True, "f16", "f16", "f16", 24),
    (17, None, 1, 672, 264, 32, True, "bf16", "bf16", "bf16", 0),
    (33, None, 1, 512, 72, 64, False, "f16", "f16", "f32", 0),
    (64, None, 1, 1152, 16, 128, False, "bf16", "f16", "f16", 8),
    (65, None, 1, 1056, 512, 32, False, "f16", "bf16", "f32", 0),
    (200, None, 1, 896, 520, 128, True, "bf16", "bf16", "f32", 0),
    (513, None, 1, 576, 1032, 64, True, "f16", "f16", "bf16", 8),
    (8, "one", 40, 512, 96, 128, False, "f16", "f16", "f16", 0),
    (8, "one", 300, 160, 64, 32, True, "bf16", "bf16", "f32", 0),
    (70, "ragged", 9, 320, 80, 64, True, "f16", "bf16", "f32", 8),
    (300, "ragged", 130, 256, 48, 128, False, "bf16", "f16", "bf16", 0),
    (1500, "ragged", 5, 384, 320, 128, True, "f16", "f16", "f32", 0),
    (700, "ragged", 7, 416, 328, 32, True, "bf16", "f16", "f16", 8),
    (130, "last", 64, 192, 32, 64, False, "f16", "f16", "f32", 0),
    (2100, "ragged", 3, 448, 776, 64, False, "bf16", "bf16", "f32", 0),
]


def _weight(E, N, K, G, zeros, s_dt, g, whole=False):
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    if whole:  # powers of two from 1 to 1/4
        scale = 2.0 ** -torch.randint(0, 3, (E, N, K // G), generator=g).float()
    else:
        scale = (torch.rand(E, N, K // G, generator=g) + 0.5) / (4.6 * K ** 0.5)
        scale *= torch.randint(0, 2, scale.shape, generator=g) * 2 - 1
    scale = scale.to(DT[s_dt])
    zero = torch.randint(0, 16, (E, N, K // G), generator=g, dtype=torch.uint8) if zeros else None
    dev = exl3.DeviceW4(q.to(DEV), scale.to(DEV), None if zero is None else zero.to(DEV))
    return dev, (q.numpy(), scale.double().numpy(), None if zero is None else zero.numpy())


@pytest.mark.parametrize("case", W4)
def test_w4_linear(case):
    _say("w4", *case)
    rows, kind, E, K, N, G, zeros, x_dt, s_dt, o_dt, pad = case
    g = torch.Generator().manual_seed(rows + N)
    W, host = _weight(E, N, K, G, zeros, s_dt, g)
    off = _offsets(kind, rows, E, g)
    x = _wide(torch.randn(rows, K, generator=g), pad, DT[x_dt])
    out = torch.full((rows, N + pad), MARK, dtype=DT[o_dt], device=DEV)
    exl3.exl3_w4_linear(x, W, None if off is None else off.to(DEV), out=out[:, :N])
    w, xn = ow4.weights(*host), _np(x)
    o = None if off is None else off.numpy()
    held = np.full((rows, N), MARK)
    ref = ow4.linear(xn, w, o, held)
    mag = ow4.linear(np.abs(xn), np.abs(w), o)
    _within(_np(out[:, :N]), ref, DT[o_dt], (2 * K + K // G) * U, mag)
    assert (out[:, N:] == MARK).all()
    if off is not None:
        assert (out[int(off[-1]):] == MARK).all()


@pytest.mark.parametrize("case", W4)
def test_w4_whole_numbers(case):
    """x of -8 .. 8 and scales that are powers of two: every partial sum is a
    multiple of 1/4 below 2^20, exact in fp32."""
    rows, kind, E, K, N, G, zeros, x_dt, s_dt, _, pad = case
    g = torch.Generator().manual_seed(rows + N + 1)
    W, host = _weight(E, N, K, G, zeros, s_dt, g, whole=True)
    off = _offsets(kind, rows, E, g)
    x = _wide(torch.randint(-8, 9, (rows, K), generator=g).float(), pad, DT[x_dt])
    out = torch.full((rows, N), MARK, device=DEV)
    exl3.exl3_w4_linear(x, W, None if off is None else off.to(DEV), out=out)
    ref = ow4.linear(_np(x), ow4.weights(*host), None if off is None else off.numpy(),
                     np.full((rows, N), MARK))
    assert np.array_equal(_np(out), ref)


# Sizes that the kernels' forms are chosen for: tiles of 128 x 256, 64 x 256,
# 32 x 128, 32 x 64, 16 x 128, 16 x 64 and 16 x 16.
FORMS = [(5000, 24, 2056), (2700, 64, 1032), (1100, 64, 1032), (700, 32, 520), (330, 64, 1032),
         (70, 33, 520), (60, 9, 328)]


def _spread(rows, E, g):
    """Offsets of experts of about rows / E rows each, some of them empty."""
    e = torch.randint(0, E, (rows,), generator=g)
    e[e == E // 2] = 0
    return torch.cat([torch.zeros(1, dtype=torch.int64),
                      torch.bincount(e, minlength=E).cumsum(0)]).to(torch.int32)


@pytest.mark.parametrize("rows,E,N", FORMS)
@pytest.mark.parametrize("K,G,zeros,x_dt,o_dt", [
    (384, 128, False, "f16", "f16"), (256, 128, True, "bf16", "f32"),
    (320, 64, True, "bf16", "bf16"), (576, 64, False, "f16", "f32"),
    (160, 32, True, "f16", "f32"), (352, 32, False, "bf16", "f16"), (32, 32, True, "bf16", "f32")])
def test_w4_forms(rows, E, N, K, G, zeros, x_dt, o_dt):
    _say("form", rows, E, N, K, G, zeros, x_dt, o_dt)
    g = torch.Generator().manual_seed(rows + K)
    W, host = _weight(E, N, K, G, zeros, "bf16" if zeros else "f16", g)
    off = _spread(rows, E, g)
    x = _wide(torch.randn(rows + 5, K, generator=g), 8, DT[x_dt])
    out = torch.full((rows + 5, N + 8), MARK, dtype=DT[o_dt], device=DEV)
    exl3.exl3_w4_linear(x, W, off.to(DEV), out=out[:, :N])
    w, xn, o = ow4.weights(*host), _np(x), off.numpy()
    ref = ow4.linear(xn, w, o, np.full((rows + 5, N), MARK))
    mag = ow4.linear(np.abs(xn), np.abs(w), o)
    _within(_np(out[:, :N]), ref, DT[o_dt], (2 * K + K // G) * U, mag)
    assert (out[:, N:] == MARK).all() and (out[rows:] == MARK).all()


@pytest.mark.parametrize("rows,E,N", FORMS[:6])
@pytest.mark.parametrize("K,G,x_dt", [(384, 128, "f16"), (320, 64, "bf16"), (352, 32, "f16")])
def test_w4_forms_give_the_same_bytes(rows, E, N, K, G, x_dt):
    """Rows of a few experts of a large call, alone: another form, the same bytes.
    Rows that hold infinities and NaN leave the others as they are."""
    g = torch.Generator().manual_seed(rows + G)
    W, _ = _weight(E, N, K, G, True, "f16", g)
    off = _spread(rows, E, g)
    x = torch.randn(rows, K, generator=g).to(DT[x_dt]).to(DEV)
    f32 = torch.float32
    full = exl3.exl3_w4_linear(x, W, off.to(DEV), f32)
    for lo, hi in ((0, 1), (int(off[1]) - 3, int(off[1]) + 20), (rows // 2, rows // 2 + 200),
                   (rows - 40, rows)):
        lo, hi = max(lo, 0), min(hi, rows)
        part = exl3.exl3_w4_linear(x[lo:hi], W, (off - lo).clamp(0, hi - lo).to(DEV), f32)
        assert _same(part, full[lo:hi]), (lo, hi)
    x[1, K - 1], x[rows // 2, 0] = float("nan"), float("inf")
    got = exl3.exl3_w4_linear(x, W, off.to(DEV), f32)
    rest = [r for r in range(rows) if r not in (1, rows // 2)]
    assert _same(got[rest], full[rest])
    assert got[1].isnan().all() and not got[rows // 2].isfinite().any()


@pytest.mark.parametrize("x_dt,G,zeros,K", [("f16", 128, False, 1664), ("bf16", 32, True, 1184),
                                            ("f16", 64, True, 1088), ("bf16", 128, True, 2176)])
def test_w4_rows_are_independent_of_their_company(x_dt, G, zeros, K):
    """A row's bytes: alone, in chunks of any length, in other orders, with its
    expert's rows elsewhere."""
    g = torch.Generator().manual_seed(K)
    rows, E, N = 2600, 4, 328
    W, _ = _weight(E, N, K, G, zeros, "f16", g)
    x = torch.randn(rows, K, generator=g).to(DT[x_dt]).to(DEV)
    f32 = torch.float32
    off = torch.tensor([0, 700, 700, 2500, rows], dtype=torch.int32, device=DEV)
    full = exl3.exl3_w4_linear(x, W, off, f32)
    for lo, hi in ((0, 1), (3, 5), (16, 32), (100, 117), (64, 128), (700, 829), (1000, 1300),
                   (701, 1700), (2499, 2502), (2500, 2600)):
        o = (off - lo).clamp(0, hi - lo)
        assert _same(exl3.exl3_w4_linear(x[lo:hi], W, o, f32), full[lo:hi]), (lo, hi)
    perm = torch.cat([torch.randperm(700, generator=g), 700 + torch.randperm(1800, generator=g),
                      torch.arange(2500, rows)]).to(DEV)
    assert _same(exl3.exl3_w4_linear(x[perm], W, off, f32), full[perm])


def test_w4_special_values():
    """An infinite or NaN row of x reaches its own outputs, a scale its own
    column, of its own expert."""
    g = torch.Generator().manual_seed(5)
    rows, K, N, G = 50, 256, 48, 64
    for x_dt in ("f16", "bf16"):
        W, host = _weight(2, N, K, G, True, "f16", g)
        off = torch.tensor([0, 20, rows], dtype=torch.int32, device=DEV)
        x = torch.randn(rows, K, generator=g).to(DT[x_dt]).to(DEV)
        clean = exl3.exl3_w4_linear(x, W, off)
        x[3, 9], x[30, 255] = float("nan"), float("inf")
        got = exl3.exl3_w4_linear(x, W, off)
        rest = [r for r in range(rows) if r not in (3, 30)]
        assert _same(got[rest], clean[rest])
        assert got[3].isnan().all()
        with np.errstate(invalid="ignore"):
            ref = _np(x)[30:31] @ ow4.weights(*host)[1].T  # inf times 0 is NaN
        ref = ref.reshape(-1)
        assert np.array_equal(np.isnan(_np(got[30])), np.isnan(ref))
        assert np.array_equal(_np(got[30])[~np.isnan(ref)], ref[~np.isnan(ref)])


def test_w4_largest_and_smallest_values():
    """Values at the ends of the types: the sums leave fp16's range, not
    fp32's; subnormal x and scales count in full."""
    K, N = 128, 16
    q = torch.full((1, N, K // 2), 0xFF, dtype=torch.uint8, device=DEV)
    x = torch.full((2, K), 65504.0, device=DEV).half()
    x[1] = 2.0 ** -24
    for s in (65504.0, 2.0 ** -24):
        W = exl3.DeviceW4(q, torch.full((1, N, 1), s, device=DEV).half())
        got = exl3.exl3_w4_linear(x, W, out_dtype=torch.float32)
        want = torch.tensor([[65504.0 * s * 7 * K], [2.0 ** -24 * s * 7 * K]], device=DEV)
        assert torch.equal(got, want.expand(2, N))
    xb = torch.full((1, K), 2.0 ** -133, dtype=torch.bfloat16, device=DEV)
    W = exl3.DeviceW4(q, torch.full((1, N, 1), 1.0, device=DEV).to(torch.bfloat16))
    got = exl3.exl3_w4_linear(xb, W, out_dtype=torch.float32)
    assert torch.equal(got, torch.full((1, N), 2.0 ** -133 * 7 * K, device=DEV))


def test_w4_strange_offsets():
    """Offsets outside the rows are clamped; ranges that descend are empty.
    Nothing outside the call's rows is written."""
    g = torch.Generator().manual_seed(6)
    rows, K, N, E = 40, 128, 32, 4
    W, host = _weight(E, N, K, 64, False, "f16", g)
    w = ow4.weights(*host)
    x = torch.randn(rows, K, generator=g).half().to(DEV)
    for off in ([-5, 10, 20, 30, 99], [0, 30, 10, 10, 25], [7, 7, 7, 7, 7],
                [2 ** 31 - 1, -2 ** 31, 0, 40, 40], [0, 0, 0, 0, -1]):
        buf = torch.full((rows + 40, N), MARK, device=DEV)
        exl3.exl3_w4_linear(x, W, torch.tensor(off, dtype=torch.int32, device=DEV),
                            out=buf[20:20 + rows])
        got = _np(buf)
        assert (got[:20] == MARK).all() and (got[20 + rows:] == MARK).all()
        o = [min(max(v, 0), rows) for v in off]
        for r in range(rows):
            mine = [e for e in range(E) if o[e] <= r < o[e + 1]]
            if not mine:
                assert (got[20 + r] == MARK).all()
            else:
                ref = [w[e] @ _np(x)[r] for e in mine]
                ok = [np.allclose(got[20 + r], v, atol=1e-4) for v in ref]
                assert any(ok) or (len(mine) > 1 and (got[20 + r] == MARK).all())


def test_w4_rows_at_a_large_distance():
    """Element offsets past 2^32 in x and out, a row's distance 2^19."""
    g = torch.Generator().manual_seed(8)
    rows, K, N, ld = 9001, 64, 24, 1 << 19
    W, _ = _weight(1, N, K, 32, True, "bf16", g)
    x = torch.randn(rows, K, generator=g).half().to(DEV)
    want = exl3.exl3_w4_linear(x, W)
    fx = torch.empty(rows, ld, dtype=torch.float16, device=DEV)
    fx[:, :K] = x
    fo = torch.empty(rows, ld, dtype=torch.float16, device=DEV)
    assert _same(exl3.exl3_w4_linear(fx[:, :K], W, out=fo[:, :N]), want)


def test_w4_rows_farther_apart_than_tiles_take():
    """Row distances from 2^23 on leave the 32-bit offsets within a tile."""
    g = torch.Generator().manual_seed(9)
    rows, K, N = 40, 192, 4104
    W, _ = _weight(1, N, K, 64, True, "f16", g)
    x = torch.randn(rows, K, generator=g).half().to(DEV)
    want = exl3.exl3_w4_linear(x, W)
    for ld in ((1 << 23) - 8, 1 << 23):
        far = torch.empty(rows, ld, dtype=torch.float16, device=DEV)
        far[:, :K] = x
        assert _same(exl3.exl3_w4_linear(far[:, :K], W), want), ld
        del far


# ------------------------------------------------- streams, graphs, devices
def _step(seed, T=90, k=3, E=8, H=256, I=192):
    g = torch.Generator().manual_seed(seed)
    f = torch.float16
    return dict(T=T, k=k, E=E, x=torch.randn(T, H, generator=g).to(f).to(DEV),
                logits=torch.randn(T, E, generator=g).to(DEV),
                dout=torch.randn(T, H, generator=g).to(f).to(DEV),
                xs=torch.zeros(T * k, H, dtype=f, device=DEV),
                dy=torch.zeros(T * k, H, dtype=f, device=DEV),
                h=torch.zeros(T * k, 2 * I, dtype=f, device=DEV),
                y=torch.zeros(T * k, H, dtype=f, device=DEV))


@pytest.fixture(scope="module")
def weights():
    g = torch.Generator().manual_seed(77)
    return (_weight(8, 384, 256, 64, True, "f16", g), _weight(8, 256, 192, 32, False, "f16", g))


def _layer(s, weights):
    """Router, rows to 4-bit experts and back, and the gradients of the routing."""
    (up, _), (down, _) = weights
    mask = torch.arange(s["T"], device=DEV) < s["T"] - 3
    ids, w = exl3.exl3_route_topk(s["logits"], s["k"], row_mask=mask)
    meta = exl3.exl3_route_pack(ids, w, s["E"])
    off = meta["expert_offset"]
    xs = exl3.exl3_permute(s["x"], meta, s["k"], out=s["xs"])
    h = exl3.exl3_w4_linear(xs, up, off, out=s["h"])
    I = h.shape[1] // 2
    a = torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()
    y = exl3.exl3_w4_linear(a.half(), down, off, out=s["y"])
    out = exl3.exl3_unpermute(y, meta, s["k"], w)
    dy, dw = exl3.exl3_unpermute_backward(s["dout"], meta, s["k"], y, w, dy=s["dy"])
    dl = exl3.exl3_route_backward(s["logits"], ids, dw)
    return dict(ids=ids, w=w, xs=xs, h=h, a=a.half(), y=y, out=out, dy=dy, dw=dw, dl=dl,
                pos=meta["pos_of_pair"], off=off)


def test_a_layer_of_4_bit_experts(weights):
    """One pass through all of them as a program would make it, each step against
    its oracle on the inputs that it was given."""
    s = _step(1)
    r = _layer(s, weights)
    T, k = s["T"], s["k"]
    pos, off = r["pos"].cpu().numpy().reshape(T, k), r["off"].cpu().numpy()
    kept = int(off[-1])
    assert kept == (T - 3) * k
    f16 = torch.float16
    assert np.array_equal(_np(r["xs"]), operm.permute(_np(s["x"]), pos, np.zeros((T * k, 256))))
    for a, y, (_, host), G in (("xs", "h", weights[0], 64), ("a", "y", weights[1], 32)):
        w, xn = ow4.weights(*host), _np(r[a])
        K = xn.shape[1]
        _within(_np(r[y])[:kept], ow4.linear(xn, w, off)[:kept], f16, (2 * K + K // G) * U,
                ow4.linear(np.abs(xn), np.abs(w), off)[:kept])
    yn, wn = _np(r["y"]), _np(r["w"])
    _within(_np(r["out"]), operm.unpermute(yn, pos, wn), f16, k * U,
            operm.unpermute(np.abs(yn), pos, wn))
    assert not r["out"][T - 3:].any()
    rdy, rdw = operm.unpermute_backward(_np(s["dout"]), yn, pos, wn, np.zeros((T * k, 256)))
    _within(_np(r["dy"]), rdy, f16, U, np.abs(rdy))
    _, mag = operm.unpermute_backward(np.abs(_np(s["dout"])), np.abs(yn), pos, wn, rdy)
    _within(_np(r["dw"]), rdw, torch.float32, 17 * U, mag)
    dl = orouter.backward(_np(s["logits"]), r["ids"].cpu().numpy(), _np(r["dw"]))
    assert np.max(np.abs(_np(r["dl"]) - dl)) <= 1e-5 * max(1.0, np.max(np.abs(dl)))


def test_two_streams_at_once(weights):
    steps = [_step(1), _step(2, T=700)]
    ref = [{n: t.clone() for n, t in _layer(s, weights).items()} for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [None, None]
        for i, st in enumerate(streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got[i] = _layer(steps[i], weights)
        torch.cuda.synchronize()
        for r, q in zip(ref, got):
            kept = int(r["off"][-1])
            for n in r:
                a, b = (r[n], q[n]) if n != "a" else (r[n][:kept], q[n][:kept])
                assert torch.equal(a, b), n


def test_graph_capture_and_replay(weights):
    s, other = _step(3), _step(4)
    for k in (s, other):
        _layer(k, weights)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(s, weights)
    for seed in (3, 5, 6, 7):
        new = _step(seed)
        for n in ("x", "logits", "dout"):
            s[n].copy_(new[n])
        want = {n: t.clone() for n, t in _layer(new, weights).items()}
        _layer(other, weights)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(out[n], want[n]), (seed, n)


def test_host_tensors_rows_zero_and_names(weights):
    x = torch.zeros(4, 16)
    meta = {"pos_of_pair": torch.zeros(8, dtype=torch.int32, device=DEV)}
    for call in (lambda: exl3.exl3_permute(x, meta, 2),
                 lambda: exl3.exl3_unpermute(torch.zeros(8, 16), meta, 2),
                 lambda: exl3.exl3_unpermute_backward(x, meta, 2),
                 lambda: exl3.exl3_w4_linear(torch.zeros(4, 256).half(), weights[0][0],
                                             torch.zeros(9, dtype=torch.int32, device=DEV))):
        with pytest.raises(exl3.Exl3Error, match="status -5"):
            call()
    e = torch.empty(0, 256, dtype=torch.float16, device=DEV)
    none = {"pos_of_pair": torch.empty(0, dtype=torch.int32, device=DEV)}
    assert exl3.exl3_permute(e, none, 2).shape == (0, 256)
    assert exl3.exl3_unpermute(e, none, 2).shape == (0, 256)
    dy, dw = exl3.exl3_unpermute_backward(e, none, 2, e)
    assert dy.shape == (0, 256) and dw.shape == (0, 2)
    off = torch.zeros(9, dtype=torch.int32, device=DEV)
    assert exl3.exl3_w4_linear(e, weights[0][0], off).shape == (0, 384)
    with exl3.Profile(16) as p:
        _layer(_step(1), weights)
    assert [n for n, _ in p.records if n != "route_pack"] == [
        "route_topk", "permute", "w4", "w4", "unpermute", "unpermute_backward", "route_backward"]
