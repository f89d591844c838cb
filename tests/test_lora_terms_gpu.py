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
