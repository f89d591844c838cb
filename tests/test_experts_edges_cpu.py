"""CPU checks of calls at the edges of what is documented for the operators that
carry rows to experts and back and for the products with 4-bit weights: empty
batches, which packed rows are read, weights in strange places."""

import pytest

torch = pytest.importorskip("torch")

from trellis_quantized_moe_amd import exl3  # noqa: E402


@pytest.mark.parametrize("topk", [1, 8])
def test_an_empty_batch_with_the_buffers_of_route_pack(monkeypatch, topk):
    """No rows, on the way that a program takes: alloc_meta's buffers hold at
    least one element each."""
    monkeypatch.setattr(exl3, "_stream", lambda: None)
    meta = exl3.alloc_meta(0, topk, 4, "cpu")
    assert meta["pos_of_pair"].numel() == 1
    meta = exl3.exl3_route_pack(torch.zeros(0, topk, dtype=torch.int32), torch.zeros(0, topk), 4,
                                meta)
    e = torch.zeros(0, 16)
    xs = exl3.exl3_permute(e, meta, topk)
    assert xs.shape == (0, 16)
    assert exl3.exl3_unpermute(xs, meta, topk, torch.zeros(0, topk)).shape == (0, 16)
    dy, dw = exl3.exl3_unpermute_backward(e, meta, topk, xs, torch.zeros(0, topk))
    assert dy.shape == (0, 16) and dw.shape == (0, topk)
    for t in (torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(exl3.Exl3Error, match="pos_of_pair"):
            exl3.exl3_permute(e, {"pos_of_pair": t}, topk)
