"""GPU: adapters whose values lie at the ends of their type's range, against
the definition in float64 (MI355X only)."""

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
