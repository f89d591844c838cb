"""GPU: the balance loss and the gradient of the routing where they can go
wrong: values that take experts or rows out, experts named more than once,
rows among others, more rows than one pass of a launch (MI355X only)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_operators_gpu as base  # noqa: E402
from oracle import router as orouter  # noqa: E402
from trellis_quantized_moe_amd import exl3  # noqa: E402

pytestmark = pytest.mark.gpu
DEV, U, DT = base.DEV, base.U, base.DT
_np, _ids, _say, _within = base._np, base._ids, base._say, base._within

inf, nan, low = float("inf"), float("nan"), float(torch.finfo(torch.float32).min)
# No two values of a row lie 80 to 120 apart (but for those far apart): between
# them exp leaves fp32's normal range, and such a t may count as 0.
SPECIAL = [
    [-inf] * 8, [nan] * 8, [-inf, 1, -inf, -inf, -inf, -inf, -inf, 0],
    [nan, 1, nan, 2, -inf, -inf, 0, -inf], [inf, 0, inf, 1, 2, 3, 4, 5],
    [low] * 8, [low, 1, low, low, low, low, low, low], [-200, -210, -240] + [-400] * 5,
    [50, 40, 30, 20, 0, 0, 0, 0], [0.0] * 8, [-0.0, 0.0, -0.0, 0.0] * 2,
    [low, inf, nan, -inf, 3, 3, 3, 3], [2e38, -2e38, 3e38, 0, 1, 1, 1, 1],
    [-1, -2, -3, -4, -5, -6, -7, -8], [-inf, nan, -30, -31, -32, -33, -34, -35]]


def _special(E, seed):
    """SPECIAL's rows at eight experts of E, the others without a part, among
    rows of ordinary values above and below zero; 4 consecutive rows share a
    wave."""
    g = torch.Generator().manual_seed(seed)
    l = torch.full((len(SPECIAL), E), -inf)
    at = torch.randperm(E, generator=g)[:8].sort().values
    l[:, at] = torch.tensor(SPECIAL, dtype=torch.float32)
    l[::2, (at[0] + 1) % E if E > 8 else at[0]] = nan if E > 8 else l[::2, at[0]]
    some = torch.randn(24, E, generator=g)
    some[8:16] = some[8:16] * 3 - 30  # waves whose rows all lie below zero
    some[17] -= 20
    l = torch.cat([l, some])
    return l[torch.randperm(l.shape[0], generator=g)] if seed else l


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 70, 260])
@pytest.mark.parametrize("seed", [0, 1])
def test_special_values_in_balance_and_gradient(E, scoring, seed):
    _say("special", E, scoring, seed)
    l = _special(E, seed)
    ids, _ = exl3.exl3_route_topk(l.to(DEV), 4, scoring)
    ids[0], ids[1, 0] = torch.tensor([0, 1, 2, 3]), 5  # named, part or no part
    ids[-1], ids[-2, 1] = -1, E + 3
    ln, iN = l.double().numpy(), _ids(ids)
    bal = exl3.exl3_balance_loss(l.to(DEV), ids, scoring, 0.4)
    ref = orouter.balance(ln, iN, scoring, 0.4)
    assert np.array_equal(_ids(bal["count"]), ref["count"])
    assert int(bal["tokens"]) == ref["tokens"]
    rel = max(base._row_rel(r, E) for r in orouter.clean(ln)) + U * 80
    _within(_np(bal["prob"]), ref["prob"], torch.float32, rel)
    _within(_np(bal["loss"]), np.array([ref["loss"]]), torch.float32, rel + 20 * U)
    dw = torch.randn(l.shape[0], 4, generator=torch.Generator().manual_seed(7))
    for renorm in (True, False):
        for use_w, use_b in ((True, True), (True, False), (False, True)):
            got = exl3.exl3_route_backward(l.to(DEV), ids, dw.to(DEV) if use_w else None, scoring,
                                           renorm, 1.3, bal if use_b else None, 0.4)
            n = dw.double().numpy() if use_w else None
            want = orouter.backward(ln, iN, n, scoring, renorm, 1.3, use_b, 0.4)
            mag = base._grad_magnitude(ln, iN, n, scoring, renorm, 1.3, 0.4, 1.0,
                                       ref["count"] if use_b else None, ref["tokens"])
            _within(_np(got), want, torch.float32, rel + 40 * U, mag)


@pytest.mark.parametrize("k", [2, 3, 15, 16, 17, 32])
@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False),
                                            ("sigmoid", True), ("sigmoid", False)])
def test_experts_named_more_than_once(k, scoring, renorm):
    """Every pair of places of a row once, a row with one expert throughout,
    rows that name none twice between them."""
    _say("twice", k, scoring, renorm)
    E, g = 70, torch.Generator().manual_seed(k)
    pairs = [(i, j) for i in range(k) for j in range(i)]
    rows = 2 * len(pairs) + 1
    l = torch.randn(rows, E, generator=g)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(rows)]).to(torch.int32)
    for n, (i, j) in enumerate(pairs):
        ids[2 * n, i] = ids[2 * n, j]
    ids[-1] = 3
    dw = torch.randn(rows, k, generator=g)
    got = exl3.exl3_route_backward(l.to(DEV), ids.to(DEV), dw.to(DEV), scoring, renorm, 1.3)
    ln, iN, n = l.double().numpy(), _ids(ids), dw.double().numpy()
    want = orouter.backward(ln, iN, n, scoring, renorm, 1.3)
    mag = base._grad_magnitude(ln, iN, n, scoring, renorm, 1.3, 0, 0, None, 0)
    rel = max(base._row_rel(r, E) for r in ln) + U * (4 * 2 + 40 + k)
    _within(_np(got), want, torch.float32, rel, mag)


MANY = 2 * 16384 + 5  # more than two passes of the largest launch


@pytest.mark.parametrize("E,k,scoring,dt", [
    (12, 3, "softmax", "f32"), (65, 17, "sigmoid", "f32"), (65, 3, "softmax", "bf16"),
    (12, 3, "sigmoid", "f16"), (200, 17, "softmax", "bf16")])
def test_more_rows_than_one_pass(E, k, scoring, dt):
    """Balance against the oracle; the gradient, in place too, against calls of
    rows that one pass holds (which the oracle tests cover): the same bytes."""
    _say("many rows", E, k, scoring, dt)
    g = torch.Generator().manual_seed(E + k)
    l = (1.5 * torch.randn(MANY, E, generator=g)).to(DT[dt])
    ids = torch.topk(l.float() + torch.randn(MANY, E, generator=g), min(k, E)).indices
    ids[torch.rand(MANY, generator=g) < 0.05] = -1
    ids[torch.rand(MANY, k, generator=g) < 0.02] = E
    twice = torch.rand(MANY, generator=g) < 0.1
    ids[twice, k - 1] = ids[twice, 0]
    ids[MANY - 1] = torch.arange(k)
    ids[MANY - 1, 1] = ids[MANY - 1, 0]
    dw = torch.randn(MANY, k, generator=g).to(DT[dt])
    l, dw, ids = l.to(DEV), dw.to(DEV), ids.to(torch.int32).to(DEV)
    bal = exl3.exl3_balance_loss(l, ids, scoring, 0.4)
    ref = orouter.balance(_np(l), _ids(ids), scoring, 0.4)
    assert np.array_equal(_ids(bal["count"]), ref["count"])
    assert int(bal["tokens"]) == ref["tokens"]
    # a lane's 3 rows, 2 steps over the wave's rows, 8 waves, 8 + 64 partial sums
    rel = max(base._row_rel(r, E) for r in _np(l)) + U * (3 + 2 + 8 + 8 + 64 + 2)
    _within(_np(bal["prob"]), ref["prob"], torch.float32, rel)
    _within(_np(bal["loss"]), np.array([ref["loss"]]), torch.float32, rel + U * 20)
    for renorm in (True, False):
        def grad(lo, hi, **kw):
            return exl3.exl3_route_backward(l[lo:hi], ids[lo:hi], dw[lo:hi], scoring, renorm, 1.3,
                                            bal, 0.4, **kw)
        full, buf = grad(0, MANY), l.clone()
        exl3.exl3_route_backward(buf, ids, dw, scoring, renorm, 1.3, bal, 0.4, dlogits=buf)
        i = torch.int32 if dt == "f32" else torch.int16
        assert torch.equal(buf.view(i), full.view(i))
        for lo in range(0, MANY, 9600):
            hi = min(lo + 9600, MANY)
            assert torch.equal(grad(lo, hi).view(i), full[lo:hi].view(i)), (renorm, lo)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_rows_are_the_same_bytes_in_any_company(scoring):
    """Rows that take another path (below zero throughout, an infinite
    gradient, an expert named twice) change nothing in the rows beside them."""
    g = torch.Generator().manual_seed(21)
    rows, E, k = 64, 70, 4
    l = torch.randn(rows, E, generator=g)
    l[::5] = -3 - 2 * l[::5].abs()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(rows)]).to(torch.int32)
    ids[3::7, 1] = ids[3::7, 0]
    ids[6::9] = -1
    dw = torch.randn(rows, k, generator=g)
    dw[9::16, 2] = inf
    dw[::3] = 0.0
    dw[1::6, 1] = -0.0
    l, ids, dw = l.to(DEV), ids.to(DEV), dw.to(DEV)
    bal = exl3.exl3_balance_loss(l, ids, scoring, 0.4)
    for renorm in (True, False):
        for b in (bal, None):
            for scale in (1.3, -1.3):
                full = exl3.exl3_route_backward(l, ids, dw, scoring, renorm, scale, b, 0.4)
                for step in (1, 3):
                    for lo in range(0, rows, step):
                        s = slice(lo, lo + step)
                        part = exl3.exl3_route_backward(l[s], ids[s], dw[s], scoring, renorm,
                                                        scale, b, 0.4)
                        assert torch.equal(part.view(torch.int32), full[s].view(torch.int32)), (
                            renorm, b is None, scale, lo, step)
