"""CPU: what the binding of the router and adapter operators refuses, because
the C ABI, given bare pointers and 32-bit sizes, could not."""

import pytest

torch = pytest.importorskip("torch")

from trellis_quantized_moe_amd import exl3  # noqa: E402

FAR = (1 << 32) + 4  # 4 in 32 bits


def test_sizes_past_32_bits():
    """Cut off to 32 bits, only the first rows would be worked on."""
    far = torch.empty(1, dtype=torch.float16)
    logits, ids = far.expand(FAR, 1), torch.empty(1, dtype=torch.int32).expand(FAR, 1)
    one = torch.zeros(1, 1, 8, dtype=torch.float16)
    l = torch.zeros(4, 8)
    for call in (lambda: exl3.exl3_route_topk(logits, 1),
                 lambda: exl3.exl3_balance_loss(logits, ids),
                 lambda: exl3.exl3_route_backward(logits, ids, dw=logits),
                 lambda: exl3.exl3_lora(far.expand(FAR, 8), one, one.view(1, 8, 1), ids[:, 0]),
                 lambda: exl3.exl3_lora(one[0], one, far.expand(1, FAR, 1), ids[:1, 0]),
                 lambda: exl3.exl3_route_topk(l, FAR, ids=far, w=far),
                 lambda: exl3.balance_workspace_size(FAR, 8),
                 lambda: exl3.lora_workspace_size(FAR, 8, 1, 1)):
        with pytest.raises(exl3.Exl3Error, match="a size of 4294967300 is out of range"):
            call()


def test_workspaces_whose_bytes_lie_apart():
    """One byte expanded has as many elements as a workspace, and no room."""
    ws = torch.empty(1, dtype=torch.uint8).expand(1 << 24)
    x = torch.zeros(4, 64, dtype=torch.float16)
    a, b = torch.zeros(2, 8, 64, dtype=torch.float16), torch.zeros(2, 32, 8, dtype=torch.float16)
    ids = torch.zeros(4, 1, dtype=torch.int32)
    for bad in (ws, torch.empty(1 << 24, dtype=torch.uint8)[::2]):
        with pytest.raises(exl3.Exl3Error, match="ws must be contiguous"):
            exl3.exl3_lora(x, a, b, ids[:, 0], ws=bad)
        with pytest.raises(exl3.Exl3Error, match="ws must be contiguous"):
            exl3.exl3_balance_loss(torch.zeros(4, 16), ids, balance=exl3.alloc_balance(16, "cpu"),
                                   ws=bad)


def test_balance_workspace_of_the_largest_row_count():
    """Rounding the row count up to whole workgroups stays in range."""
    assert exl3.balance_workspace_size((1 << 31) - 1, 8) == exl3.balance_workspace_size(1 << 30, 8)
