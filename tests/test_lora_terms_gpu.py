"""GPU: the adapters' inner products x A^T enter the second product with all
their bits, whatever the type of the inputs and of the output (MI355X only)."""

import pytest

torch = pytest.importorskip("torch")

from oracle import lora as olora  # noqa: E402
from trellis_quantized_moe_amd import exl3  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,K,N,R,n", [
    (1, 8, 8, 1, 1), (5, 264, 72, 8, 2), (61, 520, 136, 13, 9), (70, 2056, 64, 16, 3),
    (33, 8200, 40, 12, 2), (61, 136, 72, 24, 4), (40, 4104, 264, 32, 3), (130, 256, 72, 64, 2),
    (300, 264, 136, 96, 5), (90, 640, 72, 128, 2)])
def test_lora_sums_that_base_takes_back(rows, K, N, R, n, dt, out):
    """Every partial sum is an integer below 2^24 and the result at most 100,
    so it is exact; without the last 16-bit term of x A^T it is not."""
    print("terms", rows, K, N, R, n, dt, out, flush=True)
    x, a, b, ids, base, rest = olora.cancelling(rows + R, rows, K, N, R, n)
    dev = [torch.from_numpy(v).to(DEV).to(DT[dt]) for v in (x, a, b)]
    idd, based = torch.from_numpy(ids).to(DEV), torch.from_numpy(base).float().to(DEV)
    got = exl3.exl3_lora(*dev, idd, base=based, out_dtype=DT[out])
    bad = torch.nonzero(got.cpu().double() != torch.from_numpy(rest))
    assert bad.numel() == 0, (bad[:5].tolist(), bad.shape[0])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,K,N,R", [(50, 8, 64, 1), (40, 16, 136, 2), (90, 16, 72, 4),
                                        (4100, 8456, 40, 2), (33, 8456, 40, 3)])
def test_lora_general_values_closely(rows, K, N, R, dt):
    """A row has 8 inputs that are not 0: 8 products (exact) and their sums, the
    scale, R sums of two or three terms each, base: a rounding of at most 2^-23
    each, of the sum of absolute values; terms lose 2^-23. One term less would
    lose up to 2^-12 (fp16) or 2^-18 (bf16) of an entry, over the bound."""
    print("closely", rows, K, N, R, dt, flush=True)
    g = torch.Generator().manual_seed(rows + K)
    f, n = DT[dt], 3
    x = torch.zeros(rows, K)
    at = torch.stack([torch.randperm(K, generator=g)[:8] for _ in range(rows)])
    x.scatter_(1, at, torch.randn(rows, 8, generator=g))
    x, a, b = x.to(f), torch.randn(n, R, K, generator=g).to(f), torch.randn(n, N, R, generator=g).to(f)
    scale, ids = torch.rand(n, generator=g) + 0.5, torch.randint(0, n, (rows,), generator=g)
    base = torch.randn(rows, N, generator=g)
    got = exl3.exl3_lora(x.to(DEV), a.to(DEV), b.to(DEV), ids.to(DEV), scale.to(DEV),
                         base=base.to(DEV)).cpu().numpy()
    args = [t.double().numpy() for t in (x, a, b)] + [ids.numpy(), scale.double().numpy(), None,
                                                      base.double().numpy()]
    err = abs(got - olora.lora(*args)) / olora.magnitude(*args)
    assert err.max() <= (8 + 1 + 3 * R + 1 + 1) * 2.0 ** -23
