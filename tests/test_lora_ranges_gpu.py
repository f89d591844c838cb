"""GPU: adapters whose values lie at the ends of their type's range, against
the definition in float64 (MI355X only)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from trellis_quantized_moe_amd import exl3  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("R,K", [(1, 8), (8, 264), (16, 8200), (24, 136), (64, 72), (128, 40)])
def test_lora_bf16_products_of_far_factors(R, K):
    """x A^T and B at opposite ends of fp32's range, which bf16 shares: the
    products are of ordinary size, and so are the sums. s is two products and
    exact to 2^-24, its three terms to 2^-26, the R products are summed with
    one rounding each, which the last one follows."""
    g = torch.Generator().manual_seed(R)
    rows, N, n = 40, 16, 2
    f = torch.bfloat16
    x, a = torch.zeros(rows, K), torch.zeros(n, R, K)
    x[:, 1], x[:, K - 1] = torch.rand(rows, generator=g) + 1, torch.rand(rows, generator=g) + 0.5
    a[:, :, 1] = torch.rand(n, R, generator=g) + 0.5
    a[:, :, K - 1] = torch.randn(n, R, generator=g)
    b = torch.randn(n, N, R, generator=g)
    ids = torch.arange(rows) % n
    for sx, sa, sb in ((1e-15, 1e-15, 1e35), (1e-18, 1e-18, 1e37), (1.0, 1e-30, 1e35),
                       (1e15, 1e15, 1e-35), (1.0, 1e37, 1e-36), (1e19, 1e-19, 1.0),
                       (1e-9, 1e-9, 1e22), (1e-10, 1e-10, 1e18), (1e18, 1e17, 1e-35)):
        print("far", R, K, sx, sa, sb, flush=True)
        xx, aa, bb = (sx * x).to(f), (sa * a).to(f), (sb * b).to(f)
        y = exl3.exl3_lora(xx.to(DEV), aa.to(DEV), bb.to(DEV), ids.to(DEV),
                           out_dtype=torch.float32).cpu().double()
        s = (xx.double()[:, None, :] * aa.double()[ids]).sum(2)
        mid = (xx.double().abs()[:, None, :] * aa.double()[ids].abs()).sum(2)
        ref = (s[:, None, :] * bb.double()[ids]).sum(2)
        mag = (mid[:, None, :] * bb.double()[ids].abs()).sum(2)
        assert float(mid.max()) < 2.0 ** 127 and float(mag.max()) < 2.0 ** 127
        assert float((y - ref).abs().div(mag).max()) <= (3 + 3 * R + 2) * 2.0 ** -23


def test_lora_inner_product_past_the_largest_bf16():
    """s between bf16's largest value and fp32's: finite, like its product."""
    x = torch.ones(3, 8)
    a = torch.zeros(1, 2, 8)
    a[0, 0, 0], a[0, 0, 1], a[0, 1, 0] = torch.finfo(torch.bfloat16).max, 1e36, 1.0
    b = torch.full((1, 8, 2), 2.0 ** -100)
    f = torch.bfloat16
    y = exl3.exl3_lora(x.to(f).to(DEV), a.to(f).to(DEV), b.to(f).to(DEV),
                       torch.zeros(3, dtype=torch.int32, device=DEV), out_dtype=torch.float32)
    s = float(a.to(f).double()[0, 0, :2].sum())
    assert s < float(torch.finfo(torch.float32).max)
    assert (y.double().cpu() * 2.0 ** 100 / s - 1).abs().max() <= 4 * 2.0 ** -23


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,K,R", [(1, 72, 8), (40, 72, 16), (90, 8200, 13), (33, 264, 24),
                                      (90, 72, 64), (70, 40, 128)])
def test_lora_infinite_entries(rows, K, R, dt):
    """An infinite entry of B, of an adapter that rows name: what the
    definition gives in its column (infinite, or NaN where infinities meet or
    x A^T is 0), and every other column's bytes as without it."""
    print("infinite", rows, K, R, dt, flush=True)
    inf = float("inf")
    g = torch.Generator().manual_seed(R)
    n, N = 2, 136
    f = DT[dt]
    x = torch.randn(rows, K, generator=g).to(f)
    a = torch.randn(n, R, K, generator=g).to(f)
    b = torch.randn(n, N, R, generator=g).to(f)
    ids = torch.zeros(rows, dtype=torch.long)
    ids[1::3], ids[5::11] = 1, -1
    if rows > 8:
        x[3] = 0.0  # x A^T is 0: 0 times infinity
        x[6, 2], x[8, 4] = inf, float("nan")
    plain = b.clone()
    b[0, 5, R - 1], b[0, 70, 0], b[0, 135, R // 2] = inf, -inf, inf
    b[0, 71, 0], b[0, 71, R - 1] = -inf, inf
    b[1, 64, 1], b[1, 9, R - 1], b[1, 100, 2] = -inf, inf, float("nan")
    base = torch.randn(rows, N, generator=g)
    clean, got = (exl3.exl3_lora(x.to(DEV), a.to(DEV), v.to(DEV), ids.to(DEV), base=base.to(DEV))
                  .cpu() for v in (plain, b))
    s = torch.einsum("tk,trk->tr", x.double(), a.double()[ids.clamp(min=0)])
    ref = (s[:, None, :] * b.double()[ids.clamp(min=0)]).sum(2) + base.double()
    ref = torch.where((ids >= 0)[:, None], ref, base.double())
    odd = ~torch.isfinite(b.float()).all(2)[ids.clamp(min=0)] & (ids >= 0)[:, None]
    i = torch.int32
    assert torch.equal(got.view(i)[~odd], clean.view(i)[~odd])
    assert np.array_equal(np.isnan(got[odd].numpy()), np.isnan(ref[odd].numpy()))
    some = odd & ~torch.isnan(ref)
    assert torch.equal(got[some].double(), ref[some])
