"""GPU: the router, the balance loss, their gradient and the low-rank adapters
against float64 oracles (MI355X only).

Tolerances. An output is off by at most half a step of its type (relative
eps / 2, absolute half the smallest subnormal) plus what fp32 arithmetic loses
before it:
  u = 2^-24 per rounding. exp(l - m) loses 2 |l - m| u from its argument, which
  is rounded twice, and 2 u of its own; a sum over a row adds one rounding per addition (4 I + 4
  of them: a lane's values, then four steps), divisions and products one each.
Adapter sums of small integers are exact in fp32 and in the 16-bit terms, so
those tests compare bytes; sums of general values use the rounding count of
their longest chain.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import lora as olora  # noqa: E402
from oracle import moe as omoe  # noqa: E402
from oracle import router as orouter  # noqa: E402
from trellis_quantized_moe_amd import exl3, synth  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def _say(*a):
    print(*a, flush=True)


def _np(t):
    return t.detach().cpu().double().numpy()


def _half(dt):
    return torch.finfo(dt).eps / 2


def _wide(t, pad, dtype, fill=float("nan")):
    """t as a column slice of a wider buffer of `dtype` filled with `fill`."""
    r, c = t.shape
    buf = torch.full((r, c + pad), fill, dtype=dtype, device=DEV)
    buf[:, :c] = t.to(DEV)
    return buf[:, :c]


def _within(got, ref, dt, rel, mag=None):
    """|got - ref| <= half a step + rel * mag (mag: |ref| by default), and the
    same non-finite values."""
    got, ref = np.asarray(got), np.asarray(ref)
    mag = np.abs(ref) if mag is None else mag
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
    err = np.abs(got - ref)[fin]
    tol = (np.abs(ref) * _half(dt) + TINY[dt] + rel * mag * (1 + _half(dt)))[fin]
    assert np.all(err <= tol), "max excess %.3g" % np.max(err / np.maximum(tol, 1e-300))


# ------------------------------------------------------------------- route
def _row_rel(l, E):
    """Relative error of a normalised t of a row of logits l (see above)."""
    fin = l[np.isfinite(l)]
    span = min(float(fin.max() - fin.min()), 104.0) if fin.size else 0.0
    return U * (2 * span + 4 * ((E + 63) // 64) + 4 + 12)


def _ids(t):
    return t.cpu().numpy().astype(np.int64)


@pytest.mark.parametrize("rows,E,k,dt,wdt,idt,scoring,renorm,bias,pad,mask", [
    (1, 1, 1, "f32", "f32", "i32", "softmax", True, False, 0, False),
    (1, 128, 8, "bf16", "bf16", "i64", "softmax", True, False, 0, False),
    (3, 2, 2, "f16", "f16", "i32", "softmax", False, False, 1, False),
    (17, 7, 3, "f32", "f32", "i64", "sigmoid", True, False, 0, True),
    (64, 60, 6, "bf16", "f32", "i32", "sigmoid", False, True, 4, False),
    (33, 63, 32, "f32", "f32", "i32", "softmax", True, False, 2, True),
    (16, 64, 17, "f16", "bf16", "i32", "sigmoid", True, True, 0, False),
    (15, 65, 4, "f32", "f32", "i32", "softmax", False, False, 3, False),
    (200, 129, 8, "bf16", "f16", "i32", "sigmoid", True, True, 8, True),
    (100, 192, 8, "f32", "f16", "i32", "softmax", True, False, 0, False),
    (31, 256, 16, "f32", "f32", "i64", "sigmoid", True, True, 64, False),
    (40, 257, 8, "bf16", "f32", "i32", "softmax", True, False, 0, False),
    (9, 512, 32, "f32", "f32", "i32", "softmax", False, False, 0, False),
    (9, 600, 22, "f16", "f32", "i32", "sigmoid", False, False, 0, False),
    (5, 1024, 32, "f32", "f32", "i32", "sigmoid", True, True, 0, False),
    (6, 1001, 1, "bf16", "f32", "i32", "softmax", True, False, 0, True),
    (1025, 256, 8, "f32", "f32", "i32", "sigmoid", True, True, 0, True),
    (1030, 300, 32, "bf16", "f32", "i32", "softmax", True, False, 1, False),
    (1026, 1024, 9, "f16", "f32", "i64", "sigmoid", False, True, 0, False),
])
def test_route_topk(rows, E, k, dt, wdt, idt, scoring, renorm, bias, pad, mask):
    _say("route", rows, E, k, dt, scoring, renorm, bias, pad)
    g = torch.Generator().manual_seed(rows * 1000 + E)
    l = 2 * torch.randn(rows, E, generator=g)
    if dt == "f32":
        l = (l * 8).round() / 8  # ties
    lg = _wide(l, pad, DT[dt])
    b = (0.2 * torch.randn(E, generator=g)).to(DEV) if bias else None
    m = (torch.rand(rows, generator=g) < 0.7).to(DEV) if mask else None
    ids, w = exl3.exl3_route_topk(lg, k, scoring, renorm, 1.5, b, m,
                                  torch.int64 if idt == "i64" else torch.int32, DT[wdt])
    torch.cuda.synchronize()
    ln = _np(lg)
    ri, rw = orouter.route_topk(ln, k, scoring, renorm, 1.5, None if b is None else _np(b),
                                None if m is None else m.cpu().numpy())
    assert np.array_equal(_ids(ids), ri)
    rel = max(_row_rel(r, E) for r in ln)
    _within(_np(w), rw, DT[wdt], rel)


def test_route_topk_special_values():
    """-inf, NaN, +inf, the type's lowest value, rows with fewer experts left
    than topk, rows with none; far negative sigmoid logits still share out."""
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    rows = [
        [-inf] * 8, [nan] * 8, [-inf, 1, -inf, -inf, -inf, -inf, -inf, 0],
        [nan, 1, nan, 2, -inf, -inf, 0, -inf], [inf, 0, inf, 1, 2, 3, 4, 5],
        [low] * 8, [low, 1, low, low, low, low, low, low], [-200.0, -210, -300] + [-400.0] * 5,
        [100, 90, 80, 70, 0, 0, 0, 0], [0.0] * 8, [-0.0, 0.0, -0.0, 0.0] * 2,
        [low, inf, nan, -inf, 3, 3, 3, 3], [2e38, -2e38, 3e38, 0, 1, 1, 1, 1]]
    l = torch.tensor(rows, dtype=torch.float32)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _say("special", scoring, renorm)
            ids, w = exl3.exl3_route_topk(l.to(DEV), 4, scoring, renorm)
            ri, rw = orouter.route_topk(l.numpy(), 4, scoring, renorm)
            assert np.array_equal(_ids(ids), ri)
            _within(_np(w), rw, torch.float32, U * (2 * 104 + 30))
    # biases that exclude (NaN, -inf) or force (+inf) an expert
    b = torch.tensor([nan, -inf, inf, 0.5, 0, 0, 0, 0]).to(DEV)
    z = torch.zeros(2, 8).to(DEV)
    ids, w = exl3.exl3_route_topk(z, 8, "sigmoid", True, 1.0, b)
    assert _ids(ids)[0].tolist() == [2, 3, 4, 5, 6, 7, -1, -1]
    _within(_np(w)[0], np.array([1 / 6] * 6 + [0, 0]), torch.float32, U * 8)


def test_route_topk_near_ties_with_bias():
    """Scores 1e-9 apart (below fp32's step at 0.5) are ordered by value, not
    by index."""
    E = 64
    b = torch.zeros(E)
    l = torch.zeros(4, E)
    want = []
    for e in range(E):  # sigmoid(0) + b; ascending by 1e-9 steps of l's own sigmoid
        l[:, e] = e * 4e-9
    ids, _ = exl3.exl3_route_topk(l.to(DEV), 8, "sigmoid", True, 1.0, b.to(DEV))
    want = list(range(E - 1, E - 9, -1))
    assert _ids(ids)[3].tolist() == want


@pytest.mark.parametrize("E,k,dt", [(65, 8, "f32"), (256, 8, "bf16"), (1023, 32, "f32")])
def test_route_topk_rows_are_the_same_bytes_among_few_and_many(E, k, dt):
    """Up to 1024 rows and more take rows of 64 and of 16 lanes."""
    g = torch.Generator().manual_seed(E)
    l = (2 * torch.randn(1500, E, generator=g)).to(DEV).to(DT[dt])
    l[3, ::2], l[4], l[5, 1] = float("-inf"), float("nan"), float("inf")
    b = (0.2 * torch.randn(E, generator=g)).to(DEV)
    for scoring, renorm, bias in (("softmax", True, None), ("softmax", False, None),
                                  ("sigmoid", True, b), ("sigmoid", False, None)):
        ids, w = exl3.exl3_route_topk(l, k, scoring, renorm, 1.5, bias)
        for lo, hi in ((0, 1), (1, 7), (7, 1031), (1031, 1500)):
            i, v = exl3.exl3_route_topk(l[lo:hi], k, scoring, renorm, 1.5, bias)
            assert torch.equal(i, ids[lo:hi]) and torch.equal(v, w[lo:hi]), (scoring, renorm, lo)


def test_route_topk_more_rows_than_one_axis_of_a_launch_holds():
    rows = (1 << 28) + 37  # 16 threads a row: over 2^32 threads
    l = torch.zeros(rows, 1, dtype=torch.float16, device=DEV)
    ids = torch.full((rows, 1), 7, dtype=torch.int32, device=DEV)
    without = [0, 15, (1 << 26) - 1, 1 << 28, rows - 1]
    l[without] = float("-inf")
    _, w = exl3.exl3_route_topk(l, 1, "softmax", True, 0.5, ids=ids, w_dtype=torch.float16)
    torch.cuda.synchronize()
    out = torch.nonzero(ids[:, 0] != 0).flatten()
    assert out.tolist() == without and (ids[without] == -1).all()
    w = w[:, 0]
    assert not w[without].any() and int((w == 0.5).sum()) == rows - len(without)


# ----------------------------------------------------------------- balance
ROUTED = [
    (1, 1, 1, "f32", "softmax", 0), (1, 128, 8, "bf16", "sigmoid", 0),
    (17, 7, 3, "f32", "sigmoid", 1), (300, 60, 6, "f16", "softmax", 4),
    (33, 65, 32, "f32", "softmax", 3), (5000, 192, 8, "f32", "softmax", 0),
    (700, 256, 8, "bf16", "sigmoid", 0), (50, 257, 17, "f32", "sigmoid", 0),
    (40, 1024, 8, "f32", "softmax", 8), (20, 513, 32, "bf16", "softmax", 0),
]


def _routed(rows, E, k, dt, pad, seed, bad=True):
    g = torch.Generator().manual_seed(seed)
    l = 1.5 * torch.randn(rows, E, generator=g) + torch.randn(E, generator=g)
    lg = _wide(l, pad, DT[dt])
    ids = torch.topk(lg.float(), k, dim=1).indices
    if bad and rows > 4:
        ids[1] = -1                     # rows that take no part
        ids[rows - 1] = E
        ids[2, 0] = -5                  # single entries left out
        ids[3, k - 1] = ids[3, 0]       # an expert named twice
    return lg, ids


@pytest.mark.parametrize("rows,E,k,dt,scoring,pad", ROUTED)
def test_balance_loss(rows, E, k, dt, scoring, pad):
    _say("balance", rows, E, k, dt, scoring)
    lg, ids = _routed(rows, E, k, dt, pad, rows + E)
    for idt in (torch.int32, torch.int64):
        got = exl3.exl3_balance_loss(lg, ids.to(idt), scoring, 0.37)
        again = exl3.exl3_balance_loss(lg, ids.to(idt), scoring, 0.37)
        torch.cuda.synchronize()
        ref = orouter.balance(_np(lg), _ids(ids), scoring, 0.37)
        assert np.array_equal(_ids(got["count"]), ref["count"])
        assert int(got["tokens"]) == ref["tokens"]
        # sums of positive terms: one rounding per row a lane takes, then the
        # workgroup's 6 and the workgroups'
        rel = max(_row_rel(r, E) for r in _np(lg)) + U * (rows / 16 / 256 + 1 + 6 + 256 + 2)
        _within(_np(got["prob"]), ref["prob"], torch.float32, rel)
        _within(_np(got["loss"]), np.array([ref["loss"]]), torch.float32, rel + U * 20)
        for n in got:
            assert torch.equal(got[n], again[n]), n


def test_balance_without_rows():
    lg, ids = _routed(40, 64, 4, "f32", 0, 1)
    for l, i in ((lg, torch.full_like(ids, -1)), (lg[:0], ids[:0])):
        got = exl3.exl3_balance_loss(l, i.contiguous(), "softmax", 2.0)
        assert int(got["tokens"]) == 0 and float(got["loss"]) == 0
        assert not got["prob"].any() and not got["count"].any()
        if l.shape[0]:
            d = exl3.exl3_route_backward(l, i.contiguous(), balance=got, coef=2.0)
            assert not d.any()


# ---------------------------------------------------------------- backward
def _grad_magnitude(l, ids, dw, scoring, renorm, scale, coef, dloss, count, tokens):
    """The gradient's terms added as absolute values."""
    l = orouter.clean(l)
    T, E = l.shape
    k = ids.shape[1]
    out = np.zeros((T, E))
    for t in range(T):
        at = [j for j in range(k) if 0 <= ids[t, j] < E]
        if not at:
            continue
        e = ids[t, at]
        logt = orouter._log_strength(l[t], scoring)
        p = orouter._normalised(logt)
        if dw is not None:
            d = np.abs(dw[t, at])
            if renorm:
                q = orouter._normalised(logt[e])
                np.add.at(out[t], e, abs(scale) * q * (d + np.sum(q * d)))
            elif scoring == "softmax":
                np.add.at(out[t], e, abs(scale) * p[e] * d)
                out[t] += p * abs(scale) * np.sum(p[e] * d)
            else:
                np.add.at(out[t], e, abs(scale) * np.exp(logt[e]) * d)
        if count is not None and tokens:
            f = count / (tokens * k)
            out[t] += abs(dloss * coef) * E / tokens * p * (f + np.sum(f * p))
        if scoring == "sigmoid":
            out[t] *= np.exp(-np.logaddexp(0, l[t]))
    return out


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("rows,E,k,dt,scoring,pad", ROUTED)
def test_route_backward(rows, E, k, dt, scoring, pad, renorm):
    _say("backward", rows, E, k, dt, scoring, renorm)
    lg, ids = _routed(rows, E, k, dt, pad, rows + E)
    g = torch.Generator().manual_seed(9)
    dw = torch.randn(rows, k, generator=g).to(DEV).to(DT[dt])
    dloss = torch.tensor([-1.7], device=DEV)
    ln, iN = _np(lg), _ids(ids)
    bal = exl3.exl3_balance_loss(lg, ids, scoring, 0.5)
    rel = max(_row_rel(r, E) for r in ln) + U * (4 * ((E + 63) // 64) + 40)
    for use_w, use_b, odt in ((True, True, torch.float32), (True, False, torch.float32),
                              (False, True, DT[dt])):
        got = exl3.exl3_route_backward(lg, ids.to(torch.int32), dw if use_w else None, scoring,
                                       renorm, 1.3, bal if use_b else None, 0.5, dloss,
                                       dlogits_dtype=odt)
        torch.cuda.synchronize()
        n = _np(dw) if use_w else None
        ref = orouter.backward(ln, iN, n, scoring, renorm, 1.3, use_b, 0.5, -1.7)
        mag = _grad_magnitude(ln, iN, n, scoring, renorm, 1.3, 0.5, -1.7,
                              _np(bal["count"]) if use_b else None, int(bal["tokens"]))
        _within(_np(got), ref, odt, rel, mag)


def test_route_backward_against_differences():
    """Central differences of the float64 scalar at GPU-routed IDs: the step's
    error is ~1e-9, the kernel's U times the terms (all below 4)."""
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            _say("differences", scoring, renorm)
            g = torch.Generator().manual_seed(5)
            l = torch.randn(6, 11, generator=g)
            ids, _ = exl3.exl3_route_topk(l.to(DEV), 3, scoring, renorm, 1.3)
            dw = torch.randn(6, 3, generator=g)
            bal = exl3.exl3_balance_loss(l.to(DEV), ids, scoring, 0.5)
            got = _np(exl3.exl3_route_backward(l.to(DEV), ids, dw.to(DEV), scoring, renorm, 1.3,
                                               bal, 0.5))
            x = l.double().numpy()
            args = (_ids(ids), dw.double().numpy(), scoring, renorm, 1.3, 0.5, 1.0,
                    _np(bal["count"]), int(bal["tokens"]))
            for t in range(6):
                for e in range(11):
                    hi, lo = x.copy(), x.copy()
                    hi[t, e] += 1e-5
                    lo[t, e] -= 1e-5
                    d = (orouter.loss_of_logits(hi, *args) - orouter.loss_of_logits(lo, *args))
                    assert abs(d / 2e-5 - got[t, e]) < 1e-8 + 4 * 100 * U


def test_route_backward_excluded_experts_and_in_place():
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(2)
    l = torch.randn(20, 70, generator=g)
    l[0, 3], l[0, 5], l[1, :] = -inf, nan, -inf
    l[2, 1:] = nan
    l[3, 0] = inf
    ids, _ = exl3.exl3_route_topk(l.to(DEV), 4)
    ids[1] = torch.tensor([0, 1, 2, 3])  # named although they take no part
    bal = exl3.exl3_balance_loss(l.to(DEV), ids)
    dw = torch.randn(20, 4, generator=g)
    dw[5, 2] = inf  # its own row only
    for renorm in (True, False):
        buf = l.to(DEV).clone()
        d = exl3.exl3_route_backward(l.to(DEV), ids, dw.to(DEV), renorm=renorm, balance=bal)
        exl3.exl3_route_backward(buf, ids, dw.to(DEV), renorm=renorm, balance=bal, dlogits=buf)
        assert torch.equal(d.view(torch.int32), buf.view(torch.int32))
        d = d.cpu()
        assert d[0, 3] == 0 and d[0, 5] == 0 and not d[1].any() and not d[2, 1:].any()
        keep = [r for r in range(20) if r != 5]
        assert torch.isfinite(d[keep]).all()


def test_gradient_output_slice_leaves_its_neighbours():
    lg, ids = _routed(50, 30, 3, "f32", 0, 4)
    buf = torch.full((50, 40), 7.0, device=DEV)
    exl3.exl3_route_backward(lg, ids, torch.ones(50, 3, device=DEV), dlogits=buf[:, 3:33])
    ref = exl3.exl3_route_backward(lg, ids, torch.ones(50, 3, device=DEV))
    assert torch.equal(buf[:, 3:33], ref) and (buf[:, :3] == 7).all() and (buf[:, 33:] == 7).all()


# -------------------------------------------------------------------- lora
def _ints(g, *shape, lo=-2, hi=3):
    return torch.randint(lo, hi, shape, generator=g).float()


def _pattern(g, rows, n, order):
    if order == "none":
        return torch.full((rows,), -1)
    if order == "one":
        return torch.full((rows,), n - 1)
    if order == "rows":
        return torch.randint(-1, n + 1, (rows,), generator=g)  # -1 and n: no adapter
    ends = torch.randint(0, rows + 1, (6,), generator=g).sort().values
    req = torch.searchsorted(ends, torch.arange(rows), right=True)
    return torch.randint(0, n, (7,), generator=g)[req]


LORA = [
    # rows, K, N, R, adapters, x, base, out, order, pad
    (1, 8, 8, 1, 1, "f16", "none", "f32", "one", 0),
    (1, 4096, 4096, 16, 8, "f16", "f32", "f16", "one", 0),
    (2, 40, 24, 3, 2, "bf16", "bf16", "bf16", "rows", 8),
    (16, 512, 64, 8, 3, "bf16", "f32", "f32", "rows", 0),
    (12, 264, 72, 40, 5, "f16", "f32", "bf16", "rows", 8),
    (15, 8200, 136, 12, 700, "bf16", "bf16", "f32", "rows", 0),
    (16, 136, 72, 33, 2, "bf16", "f16", "f32", "requests", 0),
    (17, 520, 72, 17, 3, "f16", "f16", "f16", "one", 0),
    (61, 2048, 192, 32, 48, "bf16", "f32", "f32", "rows", 0),
    (63, 2056, 264, 24, 2, "f16", "none", "bf16", "requests", 0),
    (64, 504, 256, 40, 1, "bf16", "bf16", "f32", "one", 16),
    (65, 1000, 320, 64, 2, "f16", "f32", "f32", "one", 0),
    (130, 256, 1032, 65, 5, "bf16", "f16", "f16", "rows", 8),
    (257, 4104, 128, 128, 4, "f16", "bf16", "f16", "requests", 0),
    (300, 640, 200, 96, 1024, "bf16", "none", "f32", "rows", 0),
    (700, 384, 136, 5, 3, "f16", "f32", "f32", "requests", 4),
    (2047, 128, 64, 16, 3, "bf16", "bf16", "bf16", "requests", 0),
    (2049, 128, 64, 16, 64, "f16", "f16", "f16", "rows", 0),
    (5000, 64, 96, 33, 7, "bf16", "f32", "f32", "rows", 0),
    (4100, 256, 128, 48, 2, "f16", "f32", "f16", "none", 0),
]


@pytest.mark.parametrize("rows,K,N,R,n,dt,base,out,order,pad", LORA)
def test_lora_exact_on_integers(rows, K, N, R, n, dt, base, out, order, pad):
    """Integer data: every sum is an integer below 2^24 and s (below 4 K <=
    2^15) fits the 16-bit terms, so the result is the exact sum rounded once."""
    _say("lora", rows, K, N, R, n, dt, base, out, order)
    g = torch.Generator().manual_seed(rows + K)
    x, a, b = _ints(g, rows, K), _ints(g, n, R, K), _ints(g, n, N, R, lo=-1, hi=2)
    scale = torch.pow(2.0, torch.randint(-1, 2, (n,), generator=g))
    ids = _pattern(g, rows, n, order)
    ranks = torch.randint(-1, R + 3, (n,), generator=g)
    bs = None if base == "none" else _ints(g, rows, N, lo=-8, hi=9)
    eff = ranks.clamp(0, R)
    inside = torch.arange(R)[None, :] < eff[:, None]
    for use_ranks in (False, True):
        aa, bb = a.clone(), b.clone()
        if use_ranks:  # what lies past an adapter's ranks is not used
            aa[~inside] = float("nan")
            bb.transpose(1, 2)[~inside] = float("nan")
        xd = _wide(x, pad * 2 if pad % 8 else pad, DT[dt])
        bd = None if bs is None else _wide(bs, pad, DT[base])
        got = exl3.exl3_lora(xd, aa.to(DEV).to(DT[dt]), bb.to(DEV).to(DT[dt]),
                             ids.to(DEV).to(torch.int32 if use_ranks else torch.int64),
                             scale=scale.to(DEV),
                             ranks=ranks.to(torch.int32).to(DEV) if use_ranks else None,
                             base=bd, out_dtype=DT[out])
        torch.cuda.synchronize()
        ok = (ids >= 0) & (ids < n)
        at = torch.where(ok, ids, 0)
        ref = torch.zeros(rows, N, dtype=torch.float64) if bs is None else bs.double().clone()
        for i in at[ok].unique().tolist():
            r = torch.nonzero(ok & (at == i)).flatten()
            e = int(eff[i]) if use_ranks else R
            ref[r] += float(scale[i]) * (x[r].double() @ a[i, :e].double().T) @ b[
                i, :, :e].double().T
        assert float(ref.abs().max()) < 2 ** 24
        want = ref.to(torch.float32).to(DT[out])
        bad = torch.nonzero(got.cpu() != want)
        assert bad.numel() == 0, (bad[:5].tolist(), bad.shape[0])


def test_lora_values_and_ranges():
    """General values, s far outside fp16's range and deep below it. Roundings:
    a slice's chain of min(K, 512) products and the slices, R terms, the output;
    each at most 2^-23 of the sum of absolute values; the 16-bit terms lose
    2^-17 of an entry (two bf16 terms) or 2^-23 of the row's largest (fp16)."""
    for dt, odt, size in (("f16", "f32", 1.0), ("f16", "f32", 200.0), ("f16", "f32", 2e-3),
                          ("bf16", "f32", 1.0), ("bf16", "bf16", 1e6), ("bf16", "f16", 1e-3),
                          ("f16", "bf16", 300.0)):
        _say("lora values", dt, odt, size)
        g = torch.Generator().manual_seed(11)
        rows, K, N, R, n = 150, 1536, 96, 24, 3
        x = (size * torch.randn(rows, K, generator=g)).to(DT[dt])
        a = (0.5 * torch.randn(n, R, K, generator=g)).to(DT[dt])
        b = torch.randn(n, N, R, generator=g).to(DT[dt])
        scale = torch.rand(n, generator=g) + 0.5
        ids = torch.randint(-1, n, (rows,), generator=g)
        base = torch.randn(rows, N, generator=g)
        got = exl3.exl3_lora(x.to(DEV), a.to(DEV), b.to(DEV), ids.to(DEV), scale.to(DEV),
                             base=base.to(DEV), out_dtype=DT[odt])
        args = [t.double().numpy() for t in (x, a, b)] + [ids.numpy(), scale.double().numpy(),
                                                          None, base.double().numpy()]
        ref, mag = olora.lora(*args), olora.magnitude(*args)
        ref[np.abs(ref) > float(torch.finfo(DT[odt]).max)] *= np.inf  # past the type's range
        terms = 2.0 ** -17 if dt == "bf16" and odt != "f32" else 2.0 ** -23
        rel = (512 + 3 + R + 4) * 2.0 ** -23 + terms
        # fp16 terms: relative to the row's largest s, at most R times over
        _within(_np(got), ref, DT[odt], rel * (R if dt == "f16" else 1), mag)


def test_lora_nan_and_inf_stay_in_their_row():
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(1)
    rows, K, N, R, n = 40, 256, 64, 16, 4
    x, a, b = _ints(g, rows, K), _ints(g, n, R, K), _ints(g, n, N, R)
    ids = torch.arange(rows) % 3
    ids[7] = -1
    base = _ints(g, rows, N)
    clean = exl3.exl3_lora(x.to(DEV).half(), a.to(DEV).half(), b.to(DEV).half(), ids.to(DEV),
                           base=base.to(DEV))
    a[3], b[3] = nan, inf  # an adapter nobody names
    x[4, 9], x[5, 0], x[7] = nan, inf, nan  # row 7 has no adapter
    for dt in (torch.float16, torch.bfloat16):
        got = exl3.exl3_lora(x.to(DEV).to(dt), a.to(DEV).to(dt), b.to(DEV).to(dt), ids.to(DEV),
                             base=base.to(DEV))
        rest = [r for r in range(rows) if r not in (4, 5)]
        assert torch.equal(got[rest], clean[rest])
        assert torch.isnan(got[4]).all() and not torch.isfinite(got[5]).any()


def test_lora_in_place_and_neighbours():
    """out = base: rows without an adapter keep their bytes (a NaN's payload
    too), columns and rows beside the slice stay as they were."""
    g = torch.Generator().manual_seed(6)
    rows, K, N, R, n = 90, 128, 200, 12, 3
    x, a, b = (_ints(g, *s).to(DEV).to(torch.bfloat16) for s in ((rows, K), (n, R, K), (n, N, R)))
    ids = torch.randint(-1, n + 1, (rows,), generator=g).to(DEV)
    ids[0] = -1
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        buf = _ints(g, rows + 4, N + 24).to(DEV).to(dt)
        view = buf[2:2 + rows, 8:8 + N]
        buf[2, 8] = float("nan")
        before = buf.clone()
        want = exl3.exl3_lora(x, a, b, ids, base=view)
        exl3.exl3_lora(x, a, b, ids, base=view, out=view)
        i = torch.int32 if dt == torch.float32 else torch.int16
        assert torch.equal(view.contiguous().view(i), want.view(i))
        none = (ids < 0) | (ids >= n)
        assert torch.equal(view[none].contiguous().view(i),
                           before[2:2 + rows, 8:8 + N][none].contiguous().view(i))
        before[2:2 + rows, 8:8 + N] = view
        assert torch.equal(buf.view(i), before.view(i))


def test_lora_rows_are_independent_of_their_company():
    """A row's bytes: alone, in other orders, among other rows, in chunks."""
    g = torch.Generator().manual_seed(8)
    rows, K, N, R, n = 2500, 4608, 136, 40, 5
    x = torch.randn(rows, K, generator=g).to(torch.bfloat16).to(DEV)
    a = torch.randn(n, R, K, generator=g).to(torch.bfloat16).to(DEV)
    b = torch.randn(n, N, R, generator=g).to(torch.bfloat16).to(DEV)
    ids = torch.randint(-1, n, (rows,), generator=g).to(DEV)
    full = exl3.exl3_lora(x, a, b, ids, out_dtype=torch.float32)
    perm = torch.randperm(rows, generator=g).to(DEV)
    mixed = exl3.exl3_lora(x[perm], a, b, ids[perm], out_dtype=torch.float32)
    assert torch.equal(mixed, full[perm])
    for lo, hi in ((0, 1), (1, 18), (700, 800), (2040, 2100), (2499, 2500)):
        part = exl3.exl3_lora(x[lo:hi], a, b, ids[lo:hi], out_dtype=torch.float32)
        assert torch.equal(part, full[lo:hi]), (lo, hi)


def test_lora_rows_are_the_same_bytes_in_one_launch_and_two():
    """Rank 16 over a long K: few rows take two launches, many take one."""
    g = torch.Generator().manual_seed(12)
    rows, K, N, R, n = 4100, 8456, 200, 13, 3
    x = torch.randn(rows, K, generator=g).half().to(DEV)
    a = torch.randn(n, R, K, generator=g).half().to(DEV)
    b = torch.randn(n, N, R, generator=g).half().to(DEV)
    ids = torch.randint(-1, n, (rows,), generator=g).to(DEV)
    with exl3.Profile(8) as p:
        full = exl3.exl3_lora(x, a, b, ids, out_dtype=torch.float32)
        part = exl3.exl3_lora(x[1900:2200], a, b, ids[1900:2200], out_dtype=torch.float32)
    assert [k for k, _ in p.records] == ["lora", "lora_a", "lora_b"]
    assert torch.equal(part, full[1900:2200])


def test_lora_ids_outside_32_bits():
    x, a, b = (torch.ones(s, device=DEV, dtype=torch.float16) for s in ((4, 8), (1, 1, 8),
                                                                         (1, 8, 1)))
    ids = torch.tensor([0, 1 << 32, -(1 << 40), 1 << 62], device=DEV)
    y = exl3.exl3_lora(x, a, b, ids)
    assert (y[0] == 8).all() and not y[1:].any()


def _far(t, ld):
    """t with its rows `ld` elements apart (what lies between is not set)."""
    buf = torch.empty(t.shape[0], ld, dtype=t.dtype, device=DEV)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


@pytest.mark.parametrize("R", [9, 24])
def test_lora_rows_at_the_largest_distance(R):
    """Byte offsets past 2^31 within a window of rows and past 2^32 in all."""
    g = torch.Generator().manual_seed(R)
    rows, K, N, n, ld = 2500, 264, 72, 4, 1 << 19
    x = torch.randn(rows, K, generator=g).half().to(DEV)
    a = torch.randn(n, R, K, generator=g).half().to(DEV)
    b = torch.randn(n, N, R, generator=g).half().to(DEV)
    ids = torch.randint(-1, n, (rows,), generator=g).to(DEV)
    base = torch.randn(rows, N, generator=g).to(DEV)
    want = exl3.exl3_lora(x, a, b, ids, base=base)
    far = _far(base, ld)
    got = exl3.exl3_lora(_far(x, ld), a, b, ids, base=far, out=far)
    assert torch.equal(got, want)


def test_router_rows_at_a_large_distance():
    """Element offsets past 2^32."""
    g = torch.Generator().manual_seed(3)
    rows, E, k, ld = 9001, 12, 3, 1 << 19
    l = torch.randn(rows, E, generator=g).to(DEV)
    far = _far(l, ld)
    ids, w = exl3.exl3_route_topk(l, k)
    for p, q in zip(exl3.exl3_route_topk(far, k), (ids, w)):
        assert torch.equal(p, q)
    bal, fbal = (exl3.exl3_balance_loss(t, ids, "softmax", 0.1) for t in (l, far))
    for key in bal:
        assert torch.equal(bal[key], fbal[key])
    want = exl3.exl3_route_backward(l, ids, w, balance=bal, coef=0.1)
    exl3.exl3_route_backward(far, ids, w, balance=bal, coef=0.1, dlogits=far)
    assert torch.equal(far, want)


# ------------------------------------------------- streams, graphs, devices
def _all_operators(s):
    """Every operator on the tensors of `s`, as one step would run them."""
    logits = exl3.exl3_lora(s["x"], s["a"], s["b"], s["aid"], base=s["logits"])
    ids, w = exl3.exl3_route_topk(logits, 4, "sigmoid", True, 2.0, s["bias"])
    bal = exl3.exl3_balance_loss(logits, ids, "sigmoid", 0.1)
    d = exl3.exl3_route_backward(logits, ids, w, "sigmoid", True, 2.0, bal, 0.1, bal["loss"])
    return [logits, ids, w, bal["loss"], bal["count"], bal["prob"], bal["tokens"], d]


def _step(seed, rows=300, E=64):
    g = torch.Generator().manual_seed(seed)
    f = torch.float16
    return dict(x=torch.randn(rows, 256, generator=g).to(f).to(DEV),
                a=torch.randn(3, 8, 256, generator=g).to(f).to(DEV) / 16,
                b=torch.randn(3, E, 8, generator=g).to(f).to(DEV),
                aid=torch.randint(-1, 3, (rows,), generator=g).to(DEV),
                logits=torch.randn(rows, E, generator=g).to(DEV),
                bias=0.1 * torch.randn(E, generator=g).to(DEV))


def test_two_streams_at_once():
    steps = [_step(1), _step(2, rows=2100)]
    ref = [_all_operators(s) for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [None, None]
        for i, st in enumerate(streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got[i] = _all_operators(steps[i])
        torch.cuda.synchronize()
        for r, q in zip(ref, got):
            assert all(torch.equal(u, v) for u, v in zip(r, q))


def test_graph_capture_and_replay():
    s, other = _step(3), _step(4)
    for k in (s, other):
        _all_operators(k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _all_operators(s)
    for seed in (3, 5, 6, 7):
        new = _step(seed)
        for n in s:
            s[n].copy_(new[n])
        want = [t.clone() for t in _all_operators(new)]  # eager work between the replays
        _all_operators(other)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want)), seed


def test_host_tensors_and_rows_zero():
    l = torch.zeros(4, 16)
    with pytest.raises(exl3.Exl3Error, match="status -5"):
        exl3.exl3_route_topk(l, 2, ids=torch.empty(4, 2, dtype=torch.int32, device=DEV))
    with pytest.raises(exl3.Exl3Error, match="status -5"):
        exl3.exl3_balance_loss(l, torch.zeros(4, 2, dtype=torch.int32, device=DEV),
                               balance=exl3.alloc_balance(16))
    e = torch.empty(0, 16, device=DEV)
    ids, w = exl3.exl3_route_topk(e, 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert exl3.exl3_route_backward(e, ids, w).shape == (0, 16)
    x = torch.empty(0, 16, device=DEV, dtype=torch.float16)
    a, b = x.new_zeros(1, 4, 16), x.new_zeros(1, 8, 4)
    assert exl3.exl3_lora(x, a, b, ids.new_zeros(0)).shape == (0, 8)


def test_timing_records_name_the_launches():
    with exl3.Profile(16) as p:
        _all_operators(_step(1))
    assert [n for n, _ in p.records] == ["lora", "route_topk", "balance", "balance_sum",
                                         "route_backward"]


# ----------------------------------------------------------------- together
def test_adapted_router_feeds_the_routed_layer():
    """A shared projection and its adapters, router logits and theirs, the
    routed layer on the IDs and weights, then loss and gradient: each against
    its oracle. Padded rows go through as zeros."""
    wl = synth.moe_workload("tiny", rows=33)
    gate, up, down = (exl3.DeviceProj(p, DEV) for p in (wl.gate, wl.up, wl.down))
    x, _, _ = exl3.device_inputs(wl, DEV)
    g = torch.Generator().manual_seed(3)
    f = torch.float16
    n, R, H, E = 3, 8, wl.hidden, wl.num_experts
    proj = (torch.randn(E, H, generator=g) / 16).to(DEV)
    ra = (torch.randn(n, R, H, generator=g) / 16).to(f).to(DEV)
    rb = (torch.randn(n, E, R, generator=g) / 3).to(f).to(DEV)
    aid = torch.randint(-1, n, (33,), generator=g).to(DEV)
    mask = torch.arange(33, device=DEV) < 30
    base = x.float() @ proj.t()
    logits = exl3.exl3_lora(x, ra, rb, aid, base=base)
    ids, w = exl3.exl3_route_topk(logits, wl.topk, row_mask=mask)
    y = exl3.exl3_moe_forward(x, ids, w, gate, up, down, 33 * wl.topk)
    bal = exl3.exl3_balance_loss(logits, ids, coef=0.01)
    d = exl3.exl3_route_backward(logits, ids, torch.ones_like(w), balance=bal, coef=0.01)
    torch.cuda.synchronize()
    ref = olora.lora(_np(x), _np(ra), _np(rb), aid.cpu().numpy(), base=_np(base))
    mag = olora.magnitude(_np(x), _np(ra), _np(rb), aid.cpu().numpy(), base=_np(base))
    _within(_np(logits), ref, torch.float32, R * (H + R + 8) * 2.0 ** -23, mag)
    ri, rw = orouter.route_topk(_np(logits), wl.topk, row_mask=mask.cpu().numpy())
    assert np.array_equal(_ids(ids), ri)
    _within(_np(w), rw, torch.float32, max(_row_rel(r, E) for r in _np(logits)))
    orc = omoe.moe_forward(wl.x, ri, _np(w), wl.gate, wl.up, wl.down, "R")
    rms = float(np.sqrt(np.mean(orc ** 2)))
    assert float(np.max(np.abs(_np(y) - orc))) <= 2e-3 * rms
    assert not y[30:].any()
    assert int(bal["tokens"]) == 30 and int(bal["count"].sum()) == 30 * wl.topk
    assert not d[30:].any()
    # sum of dw w with dw = 1 and renormalised weights is constant: the loss alone is left
    rd = orouter.backward(_np(logits), ri, None, with_balance=True, coef=0.01)
    assert np.max(np.abs(_np(d) - rd)) <= 1e-6
