"""CPU: the data of the tests of the adapters' inner products shows a term of
theirs that is left out (the terms are left out here, in float64)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import lora as olora  # noqa: E402


def _terms(s, dtype, count):
    """s as the sum of `count` rounded terms, each the rest of those before
    (s below 2^14, inside fp16's range)."""
    s = s * 2.0 ** -6
    total = torch.zeros_like(s)
    for _ in range(count):
        total = total + (s - total).to(dtype).double()
    return total * 2.0 ** 6


@pytest.mark.parametrize("dtype,needed", [(torch.float16, 2), (torch.bfloat16, 3)])
@pytest.mark.parametrize("R", [1, 8, 16, 24, 64, 128])
def test_cancelling_data_needs_every_term(R, dtype, needed):
    x, a, b, ids, base, rest = olora.cancelling(R, 9, 40, 24, R, 2)
    for v in (x, a, b):
        assert np.array_equal(torch.from_numpy(v).to(dtype).double().numpy(), v)
    assert np.array_equal(torch.from_numpy(base).float().double().numpy(), base)

    def out(count):
        y = torch.from_numpy(base).clone()
        for t, i in enumerate(ids):
            if i >= 0:
                s = torch.from_numpy(a[i] @ x[t])
                assert 2 ** 17 < float(s.min()) and float(s.max()) < 2 ** 20
                y[t] += torch.from_numpy(b[i]) @ _terms(s, dtype, count)
        return y.numpy()

    assert np.array_equal(out(needed), rest)
    rows = np.asarray(ids) >= 0
    assert rows.any() and (out(needed - 1) != rest)[rows].mean() > 0.3
