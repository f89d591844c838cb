"""GPU: edges of the operators that carry rows to experts and back and of the
products with 4-bit weights (MI355X only): values at the ends of the types, every
form of the products for one projection and over many steps, rows as far apart
as a form takes, calls longer than one launch.

Tolerance of a product: half a step of the output's type, plus u = 2^-24 of the
sum of absolute terms for each rounding before it: a matrix instruction's sums
are taken as 32 additions that may each cut off (2 u), 2 in all for every input,
and an fma a group. Everything else is compared as bytes.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

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


def _same(a, b):
    n = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.contiguous().view(n), b.contiguous().view(n))


def _far(t, ld):
    """t with its rows ld elements apart."""
    buf = torch.empty(t.shape[0], ld, dtype=t.dtype, device=DEV)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def _weight(E, N, K, G, zeros, s_dt, g):
    """Laid out, as float64 [E, N, K] on the GPU, and as DeviceW4 takes them."""
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    scale = (torch.rand(E, N, K // G, generator=g) + 0.5) / (4.6 * K ** 0.5)
    scale *= torch.randint(0, 2, scale.shape, generator=g) * 2 - 1
    scale = scale.to(DT[s_dt])
    zero = torch.randint(0, 16, (E, N, K // G), generator=g, dtype=torch.uint8) if zeros else None
    parts = [None if t is None else t.to(DEV) for t in (q, scale, zero)]
    w = ow4.weights(q.numpy(), scale.double().numpy(), None if zero is None else zero.numpy())
    return exl3.DeviceW4(*parts), torch.from_numpy(w).to(DEV), parts


# Rows and outputs of one projection for each form: tiles of 128 x 256, 64 x 256,
# 32 x 128, 32 x 64, 16 x 128, 16 x 64 and 16 x 16.
SIZES = {"128x256": (3001, 4104), "64x256": (1000, 4104), "32x128": (500, 4104),
         "32x64": (130, 4104), "16x128": (9, 65488), "16x64": (60, 4104), "16x16": (20, 4104)}


# ------------------------------------------------------- values at the ends
@pytest.mark.parametrize("form", SIZES)
@pytest.mark.parametrize("x_dt,G,K", [("bf16", 32, 160), ("f16", 64, 192), ("bf16", 128, 256)])
def test_scales_that_are_infinite_or_nan(form, x_dt, G, K):
    """A scale multiplies its group's sum: its column, and no other, gets what
    scale * sum gives, NaN where the sum is 0."""
    _say("scales", form, x_dt, G, K)
    rows, N = SIZES[form]
    g = torch.Generator().manual_seed(K)
    x = torch.randint(-4, 5, (rows, K), generator=g).to(DT[x_dt]).to(DEV)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = torch.ones(N, K // G).to(torch.bfloat16)
    f32 = torch.float32
    clean = exl3.exl3_w4_linear(x, exl3.DeviceW4(q.to(DEV), s.to(DEV)), out_dtype=f32)
    last = K // G - 1
    special = {3: (0, np.inf), 17: (last, -np.inf), 40: (1, np.nan), N - 1: (last, np.inf)}
    for n, (at, v) in special.items():
        s[n, at] = v
    q[N - 1, last * G // 2:] = 0x88  # a group of zeros
    got = exl3.exl3_w4_linear(x, exl3.DeviceW4(q.to(DEV), s.to(DEV)), out_dtype=f32)
    rest = torch.ones(N, dtype=torch.bool, device=DEV)
    rest[list(special)] = False
    assert _same(got[:, rest], clean[:, rest])
    xn, v = x.double().cpu().numpy(), ow4.weights(q.numpy()[None], np.ones((1, N, 1)))[0]
    with np.errstate(invalid="ignore"):
        for n, (at, sc) in special.items():
            t = xn[:, at * G:at * G + G] @ v[n, at * G:at * G + G]
            assert np.array_equal(got[:, n].cpu().numpy(), t * sc, equal_nan=True), n


@pytest.mark.parametrize("form", SIZES)
def test_the_largest_x_whose_sums_stay_finite(form):
    """bf16 x below 2^117: a group's sum, up to 15 * 128 times that, is below
    2^128. Sums are exact here, of one power of two times whole numbers."""
    _say("largest", form)
    rows, N = SIZES[form]
    K, G = 256, 128
    x = torch.full((rows, K), 2.0 ** 116, dtype=torch.bfloat16, device=DEV)
    x[:, G:] = -2.0 ** 116
    x[rows // 2] = 255 * 2.0 ** 109  # the last value below 2^117
    q = torch.full((N, K // 2), 0xFF, dtype=torch.uint8, device=DEV)
    zero = torch.zeros(N, 2, dtype=torch.uint8, device=DEV)
    s = torch.full((N, 2), 2.0 ** -24, device=DEV).half()
    s[:, 1] = 2.0 ** -23
    got = exl3.exl3_w4_linear(x, exl3.DeviceW4(q, s, zero), out_dtype=torch.float32)
    want = torch.full((rows, N), -15.0 * 128 * 2 ** 92, device=DEV)
    want[rows // 2] = 3 * 15.0 * 128 * 255 * 2 ** 85
    assert torch.equal(got, want)


# --------------------------------------------------------- forms and borders
@pytest.mark.parametrize("form", SIZES)
@pytest.mark.parametrize("K,G,zeros,x_dt,s_dt,o_dt", [
    (2080, 32, True, "f16", "bf16", "f32"), (6208, 64, True, "bf16", "f16", "bf16"),
    (1664, 128, False, "f16", "f16", "f16")])
def test_one_projection_over_many_steps(form, K, G, zeros, x_dt, s_dt, o_dt):
    """x and out column slices of wider buffers; small runs of rows and the first
    520 outputs alone, which take the form of 16 x 16, give the same bytes."""
    _say("projection", form, K, G)
    rows, N = SIZES[form]
    if form == "16x128":
        K = K // 1024 * 128 + K % 128  # 65488 outputs: an eighth of the steps
    g = torch.Generator().manual_seed(K + rows)
    W, w, parts = _weight(1, N, K, G, zeros, s_dt, g)
    few = exl3.DeviceW4(*[None if t is None else t[:, :520] for t in parts])
    x = _far(torch.randn(rows, K, generator=g).to(DT[x_dt]).to(DEV), K + 64)
    out = torch.full((rows, N + 8), MARK, dtype=DT[o_dt], device=DEV)
    exl3.exl3_w4_linear(x, W, out=out[:, :N])
    assert (out[:, N:] == MARK).all()
    wt = w[0].t().contiguous()
    ref, mag = x.double() @ wt, x.double().abs() @ wt.abs()
    half = torch.finfo(DT[o_dt]).eps / 2
    tol = ref.abs() * half + TINY[DT[o_dt]] + (2 * K + K // G) * U * mag * (1 + half)
    assert ((out[:, :N].double() - ref).abs() <= tol).all()
    for lo, hi in ((0, 1), (rows - 1, rows), (rows // 2, min(rows // 2 + 16, rows))):
        part = exl3.exl3_w4_linear(x[lo:hi], few, out_dtype=DT[o_dt])
        assert _same(part, out[lo:hi, :520]), (lo, hi)


@pytest.mark.parametrize("K,G,x_dt", [(384, 128, "f16"), (416, 32, "bf16")])
@pytest.mark.parametrize("counts", [[129, 160, 161, 192, 193, 128, 0, 257],
                                    [1, 600, 0, 0, 33, 65, 32, 700]])
def test_tiles_of_128_rows_that_end_anywhere(K, G, x_dt, counts):
    """Experts whose last tile has 1, 32, 33, 64, 65 and 128 rows, and single
    projections with such remainders."""
    g = torch.Generator().manual_seed(K)
    rows, N, f32 = sum(counts), 5896, torch.float32
    W, w, _ = _weight(8, N, K, G, True, "f16", g)
    x = torch.randn(rows, K, generator=g).to(DT[x_dt]).to(DEV)
    ends = np.cumsum([0] + counts)
    got = exl3.exl3_w4_linear(x, W, torch.tensor(ends, dtype=torch.int32, device=DEV), f32)
    for e, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        wt, xe = w[e].t().contiguous(), x[lo:hi].double()
        tol = (xe @ wt).abs() * U + (2 * K + K // G) * U * (xe.abs() @ wt.abs()) * (1 + U)
        assert ((got[lo:hi].double() - xe @ wt).abs() <= tol).all(), e
        off = torch.zeros(9, dtype=torch.int32, device=DEV)
        off[e + 1:] = min(16, hi - lo)  # its last rows alone
        assert _same(exl3.exl3_w4_linear(x[max(lo, hi - 16):hi], W, off, f32),
                     got[max(lo, hi - 16):hi]), e


@pytest.mark.parametrize("rest", [1, 17, 33, 65])
def test_one_projection_with_a_last_tile_of_128_rows(rest):
    g = torch.Generator().manual_seed(rest)
    rows, N, K = 2944 + rest, 4104, 320
    W, _, _ = _weight(1, N, K, 64, True, "bf16", g)
    x = torch.randn(rows, K, generator=g).to(torch.bfloat16).to(DEV)
    got = exl3.exl3_w4_linear(x, W)
    for lo in (0, 128, 2944 - 16, 2944, rows - 16):
        hi = min(lo + 16, rows)
        assert _same(exl3.exl3_w4_linear(x[lo:hi], W), got[lo:hi]), lo


@pytest.mark.parametrize("rows,N", [(40, 8200), (256, 16392), (256, 49152)])
def test_rows_as_far_apart_as_tiles_take(rows, N):
    """A row distance of 2^23 - 8 is the last that tiles of 32 x 64, 64 x 256 and
    128 x 256 address (the last row of 128 almost 2^31 bytes from the first);
    from 2^23 on these sizes take the form of 16 x 16."""
    _say("far", rows, N)
    g = torch.Generator().manual_seed(N)
    K = 96
    W, _, _ = _weight(1, N, K, 32, True, "f16", g)
    x = torch.randn(rows, K, generator=g).half().to(DEV)
    want = exl3.exl3_w4_linear(x, W)
    assert _same(want[:16], exl3.exl3_w4_linear(x[:16], W))
    for ld in ((1 << 23) - 8, 1 << 23):
        far = _far(x, ld)
        assert _same(exl3.exl3_w4_linear(far, W), want), ld
        del far


# -------------------------------------------------- longer than one launch
def test_moves_of_more_rows_than_workgroups():
    """A launch has at most 2^22 workgroups along the rows: the last five rows of
    a workgroup's width are a second trip of some. With one choice a row and
    whole numbers every value is exact."""
    T, H = (1 << 22) + 5, 520
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(-8, 9, (T, H), generator=g, device=DEV, dtype=torch.int8).half()
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)
    pos[5], pos[T - 2] = -1, -1  # their places, T - 6 and 1, keep what they held
    meta = {"pos_of_pair": pos}
    xs = exl3.exl3_permute(x, meta, 1, out=torch.full((T, H), MARK, device=DEV).half())
    kept = torch.ones(T, dtype=torch.bool, device=DEV)
    kept[[5, T - 2]] = False
    assert (xs[[T - 6, 1]] == MARK).all()
    assert torch.equal(xs.flip(0)[kept], x[kept])
    out = exl3.exl3_unpermute(xs, meta, 1)
    assert not out[~kept].any() and torch.equal(out[kept], x[kept])
    del out
    w = torch.randint(-4, 5, (T, 1), generator=g, device=DEV).half()
    dy, dw = exl3.exl3_unpermute_backward(x, meta, 1, xs, w, dw_dtype=torch.float32,
                                          dy=torch.full((T, H), MARK, device=DEV).half())
    assert (dy[[T - 6, 1]] == MARK).all()
    assert torch.equal(dy.flip(0)[kept], (x * w)[kept])
    square = torch.cat([(c.float() ** 2).sum(1, keepdim=True) for c in x.split(1 << 18)])
    assert torch.equal(dw, torch.where(kept[:, None], square, 0.0))


def test_products_of_more_tiles_than_a_launch():
    """1028 tiles of rows times 4096 of outputs in the form of 16 x 16, which rows
    2^23 apart take: a second launch has the last of them. The same bytes as
    with rows side by side, in one launch of larger tiles."""
    g = torch.Generator(device=DEV).manual_seed(2)
    E, N, K, rows = 1024, 65536, 32, 1100
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(E, N, 1, generator=g, device=DEV).half()
    W = exl3.DeviceW4(q, s)
    del q
    off = torch.arange(E + 1, dtype=torch.int32, device=DEV)
    off[1:] += rows - E  # the first expert has 77
    x = torch.randn(rows, K, generator=g, device=DEV).half()
    want = exl3.exl3_w4_linear(x, W, off)
    out = torch.full((rows, N), MARK, device=DEV).half()
    assert _same(exl3.exl3_w4_linear(_far(x, 1 << 23), W, off, out=out), want)


# ------------------------------------------------------------ empty batches
def test_a_chain_without_rows():
    """From the logits to the gradient, as a program would with an empty batch."""
    E, k, H = 8, 2, 64
    logits = torch.empty(0, E, device=DEV)
    x = torch.empty(0, H, dtype=torch.float16, device=DEV)
    W = exl3.DeviceW4(torch.zeros(E, H, H // 2, dtype=torch.uint8, device=DEV),
                      torch.ones(E, H, 1, device=DEV).half())
    ids, w = exl3.exl3_route_topk(logits, k)
    meta = exl3.exl3_route_pack(ids, w, E)
    y = exl3.exl3_w4_linear(exl3.exl3_permute(x, meta, k), W, meta["expert_offset"])
    assert exl3.exl3_unpermute(y, meta, k, w).shape == (0, H)
    dy, dw = exl3.exl3_unpermute_backward(x, meta, k, y, w)
    assert dy.shape == (0, H) and dw.shape == (0, k)
    assert exl3.exl3_route_backward(logits, ids, dw).shape == (0, E)
