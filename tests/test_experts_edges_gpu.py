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
    """Laid out, and as float64 [E, N, K] on the GPU."""
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    scale = (torch.rand(E, N, K // G, generator=g) + 0.5) / (4.6 * K ** 0.5)
    scale *= torch.randint(0, 2, scale.shape, generator=g) * 2 - 1
    scale = scale.to(DT[s_dt])
    zero = torch.randint(0, 16, (E, N, K // G), generator=g, dtype=torch.uint8) if zeros else None
    dev = exl3.DeviceW4(q.to(DEV), scale.to(DEV), None if zero is None else zero.to(DEV))
    w = ow4.weights(q.numpy(), scale.double().numpy(), None if zero is None else zero.numpy())
    return dev, torch.from_numpy(w).to(DEV)


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
