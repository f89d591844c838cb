"""CPU checks of the router, balance and adapter operators: the oracles
against closed forms and differences, and every refusal of the C ABI (nothing
here needs a GPU: pointers are numbers that fail the device check last)."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import lora as olora  # noqa: E402
from oracle import router as orouter  # noqa: E402
from trellis_quantized_moe_amd import exl3  # noqa: E402


# ------------------------------------------------------------------ oracles
@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False),
                                            ("sigmoid", True), ("sigmoid", False)])
def test_gradient_oracle_against_differences(scoring, renorm):
    rng = np.random.default_rng(3)
    T, E, k = 5, 9, 3
    l = rng.standard_normal((T, E))
    ids, _ = orouter.route_topk(l, k, scoring, renorm)
    ids[1, 2] = -1
    ids[2] = -1      # a row that takes no part
    ids[3, 1] = ids[3, 0]  # the same expert twice
    dw = rng.standard_normal((T, k))
    b = orouter.balance(l, ids, scoring, 0.3)
    args = (ids, dw, scoring, renorm, 1.7, 0.3, -0.8, b["count"], b["tokens"])
    g = orouter.backward(l, ids, dw, scoring, renorm, 1.7, True, 0.3, -0.8)
    step = 1e-5  # central differences: error ~ step^2 + 1e-16 / step
    for t in range(T):
        for e in range(E):
            hi, lo = l.copy(), l.copy()
            hi[t, e] += step
            lo[t, e] -= step
            d = (orouter.loss_of_logits(hi, *args) - orouter.loss_of_logits(lo, *args)) / (2 * step)
            assert abs(d - g[t, e]) < 1e-8


def test_router_oracle_against_sorting():
    rng = np.random.default_rng(4)
    l = np.round(rng.standard_normal((40, 12)), 1)  # ties
    ids, w = orouter.route_topk(l, 5)
    ref = np.argsort(-l, axis=1, kind="stable")[:, :5]
    assert np.array_equal(ids, ref)
    s = np.exp(np.take_along_axis(l, ref, 1))
    assert np.allclose(w, s / s.sum(1, keepdims=True), rtol=1e-14)
    l[0] = -np.inf
    l[1, 2:] = np.nan
    ids, w = orouter.route_topk(l, 5)
    assert np.all(ids[0] == -1) and np.all(w[0] == 0)
    assert np.all(ids[1, 2:] == -1) and abs(w[1].sum() - 1) < 1e-15


def test_balance_oracle_uniform_and_empty():
    E, k = 8, 2
    l = np.zeros((4, E))
    ids = np.arange(8).reshape(4, 2)
    b = orouter.balance(l, ids, coef=0.5)
    assert b["tokens"] == 4 and np.all(b["count"] == 1) and abs(b["loss"] - 0.5) < 1e-15
    b = orouter.balance(l, np.full((4, 2), -1))
    assert b["tokens"] == 0 and b["loss"] == 0 and not b["prob"].any()


def test_lora_oracle_against_dense():
    rng = np.random.default_rng(5)
    x, a, b = rng.standard_normal((6, 16)), rng.standard_normal((3, 4, 16)), rng.standard_normal(
        (3, 8, 4))
    ids = np.array([0, 2, -1, 1, 3, 2])
    scale = np.array([1.0, 0.5, -2.0])
    y = olora.lora(x, a, b, ids, scale, [4, 2, 9], np.ones((6, 8)))
    for t, i in enumerate(ids):
        ref = np.ones(8)
        if 0 <= i < 3:
            r = [4, 2, 4][i]
            ref = ref + scale[i] * (b[i][:, :r] @ a[i][:r]) @ x[t]
        assert np.allclose(y[t], ref, rtol=1e-13)


# ----------------------------------------------------------------- refusals
P = 1 << 20  # an address that is no device memory


def _router(**kw):
    d = dict(num_experts=64, topk=8, scoring=0, renorm=1, scale=1.0, bias=None)
    d.update(kw)
    return exl3.RouterC(*[d[n] for n in ("num_experts", "topk", "scoring", "renorm", "scale",
                                         "bias")])


def _route(router="default", logits=P, dt=exl3.F32, ld=64, rows=4, mask=None, ids=P,
           ids_dt=exl3.I32, w=P, w_dt=exl3.F32):
    r = _router() if router == "default" else router
    return exl3.lib().exl3_route_topk(ctypes.byref(r) if r else None, logits, dt, ld, rows, mask,
                                      ids, ids_dt, w, w_dt, None, None)


BAD_ROUTERS = [
    (dict(router=None), -1), (dict(router=_router(num_experts=0)), -7),
    (dict(router=_router(num_experts=1025)), -7), (dict(router=_router(topk=0)), -7),
    (dict(router=_router(topk=33)), -7), (dict(router=_router(num_experts=4, topk=5)), -7),
    (dict(router=_router(scoring=2)), -7), (dict(router=_router(scale=float("nan"))), -7),
    (dict(router=_router(scale=float("inf"))), -7),
    (dict(logits=None), -1), (dict(ids=None), -1), (dict(rows=-1), -7), (dict(rows=1 << 30), -7),
    (dict(dt=exl3.I32), -2), (dict(dt=0), -2), (dict(ids_dt=exl3.F32), -2),
    (dict(ld=63), -3), (dict(ld=-64), -3), (dict(ld=(1 << 32) + 4), -3),
    (dict(logits=P + 2), -4), (dict(logits=P + 1, dt=exl3.F16), -4), (dict(ids=P + 2), -4),
    (dict(ids=P + 4, ids_dt=exl3.I64), -4),
]


@pytest.mark.parametrize("kw,code", BAD_ROUTERS + [
    (dict(router=_router(bias=P)), -7), (dict(w=None), -1), (dict(w_dt=exl3.I64), -2),
    (dict(w=P + 2), -4), (dict(router=_router(scoring=1, bias=P + 2)), -4),
    (dict(), -5), (dict(router=_router(scoring=1, bias=P), mask=P + 1), -5),
    (dict(dt=exl3.BF16, ids_dt=exl3.I64, w_dt=exl3.F16, logits=P + 2), -5),
    (dict(rows=0, logits=None, ids=None, w=None), 0),
])
def test_route_topk_refusals(kw, code):
    assert _route(**kw) == code


def _balance(router="default", logits=P, dt=exl3.F32, ld=64, rows=4, ids=P, ids_dt=exl3.I32,
             coef=1.0, bal=(P, P, P, P), ws=P, ws_bytes=1 << 40):
    r = _router() if router == "default" else router
    b = exl3.BalanceC(*bal) if bal else None
    return exl3.lib().exl3_balance_loss(ctypes.byref(r) if r else None, logits, dt, ld, rows, ids,
                                        ids_dt, coef, ctypes.byref(b) if b else None, ws, ws_bytes,
                                        None, None)


@pytest.mark.parametrize("kw,code", BAD_ROUTERS + [
    (dict(bal=None), -1), (dict(bal=(P, P, P, None)), -1), (dict(bal=(None, P, P, P)), -1),
    (dict(ws=None), -1), (dict(coef=float("nan")), -7), (dict(bal=(P, P + 2, P, P)), -4),
    (dict(ws=P + 8), -4), (dict(ws_bytes=255), -6), (dict(rows=1 << 20, ws_bytes=4096), -6),
    (dict(), -5), (dict(rows=0), -5),
])
def test_balance_refusals(kw, code):
    assert _balance(**kw) == code


def _backward(router="default", logits=P, dt=exl3.F32, ld=64, rows=4, ids=P, ids_dt=exl3.I32,
              dw=P, dw_dt=exl3.F32, bal=(P, P, None, None), coef=1.0, dloss=P, out=2 * P,
              out_dt=exl3.F32, ldo=64):
    r = _router() if router == "default" else router
    b = exl3.BalanceC(*bal) if bal else None
    return exl3.lib().exl3_route_backward(ctypes.byref(r) if r else None, logits, dt, ld, rows,
                                          ids, ids_dt, dw, dw_dt, ctypes.byref(b) if b else None,
                                          coef, dloss, out, out_dt, ldo, None, None)


@pytest.mark.parametrize("kw,code", BAD_ROUTERS + [
    (dict(dw=None, bal=None), -1), (dict(out=None), -1), (dict(bal=(None, P, None, None)), -1),
    (dict(bal=(P, None, None, None)), -1), (dict(out_dt=exl3.I32), -2), (dict(dw_dt=0), -2),
    (dict(ldo=63), -3), (dict(coef=float("inf")), -7), (dict(out=2 * P + 2), -4),
    (dict(dw=P + 2), -4), (dict(dloss=P + 2), -4), (dict(bal=(P + 2, P, None, None)), -4),
    # in place: the same type and row distance only
    (dict(out=P, out_dt=exl3.F16), -7), (dict(out=P, ldo=128), -7), (dict(out=P), -5),
    (dict(), -5), (dict(dw=None), -5), (dict(bal=None), -5), (dict(dw=None, dw_dt=0), -5),
    (dict(rows=0, logits=None, ids=None, out=None), 0),
])
def test_backward_refusals(kw, code):
    assert _backward(**kw) == code


def _lora(ad="default", x=P, dt=exl3.F16, ldx=256, rows=4, ids=P, ids_dt=exl3.I32, base=P,
          base_dt=exl3.F32, ldb=128, out=2 * P, out_dt=exl3.F16, ldo=128, ws=P, ws_bytes=1 << 40,
          **kw):
    d = dict(in_features=256, out_features=128, rank=16, num_adapters=3, a=P, b=P, scale=P,
             ranks=P)
    d.update(kw)
    a = exl3.LoraC(*[d[n] for n in ("in_features", "out_features", "rank", "num_adapters", "a",
                                    "b", "scale", "ranks")]) if ad == "default" else ad
    return exl3.lib().exl3_lora(ctypes.byref(a) if a else None, x, dt, ldx, rows, ids, ids_dt,
                                base, base_dt, ldb, out, out_dt, ldo, ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ad=None), -1), (dict(a=None), -1), (dict(b=None), -1), (dict(x=None), -1),
    (dict(ids=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(rank=0), -7), (dict(rank=129), -7), (dict(num_adapters=0), -7),
    (dict(num_adapters=1025), -7), (dict(rows=-1), -7), (dict(rows=(1 << 26) + 1), -7),
    (dict(dt=exl3.F32), -2), (dict(ids_dt=exl3.F16), -2), (dict(out_dt=exl3.I32), -2),
    (dict(base_dt=0), -2), (dict(in_features=252), -3), (dict(out_features=0), -3),
    (dict(out_features=1 << 17, ldo=1 << 17, ldb=1 << 17), -3), (dict(ldx=248), -3),
    (dict(ldo=120), -3), (dict(ldb=127), -3), (dict(ldx=(1 << 19) + 8), -3),
    (dict(ldo=(1 << 19) + 8), -3), (dict(ldb=(1 << 19) + 8), -3),
    (dict(x=P + 8), -4), (dict(a=P + 8), -4), (dict(b=P + 4), -4), (dict(base=P + 8), -4),
    (dict(out=2 * P + 2), -4), (dict(ws=P + 8), -4), (dict(ldx=260), -4), (dict(ldo=132), -4),
    (dict(ldb=130), -4), (dict(ids=P + 2), -4), (dict(ids=P + 4, ids_dt=exl3.I64), -4),
    (dict(scale=P + 2), -4), (dict(ranks=P + 1), -4), (dict(ws_bytes=255), -6),
    # in place: the same type and row distance only
    (dict(out=P), -7), (dict(out=P, out_dt=exl3.F32, ldo=132), -7),
    (dict(out=P, out_dt=exl3.F32), -5),
    (dict(), -5), (dict(base=None, base_dt=0, ldb=0), -5), (dict(scale=None, ranks=None), -5),
    (dict(dt=exl3.BF16, rank=7, out_dt=exl3.F32, ldb=132), -5),
    (dict(rows=0, x=None, ws=None), 0),
])
def test_lora_refusals(kw, code):
    assert _lora(**kw) == code


def test_operator_workspace_sizes():
    L = exl3.lib()
    assert L.exl3_balance_workspace_size(-1, 8) == 0
    assert L.exl3_balance_workspace_size(8, 1025) == 0
    assert L.exl3_balance_workspace_size(0, 8) >= 256
    assert L.exl3_lora_workspace_size(7, 0, 8, 1) == 0
    assert L.exl3_lora_workspace_size(7, 4096, 129, 1) == 0
    assert L.exl3_lora_workspace_size(7, 4096, 8, 0) == 0
    assert L.exl3_lora_workspace_size((1 << 26) + 1, 4096, 8, 1) == 0
    assert L.exl3_lora_workspace_size(7, 4096, 9, 3) >= 7 * 9 * 4
    # 64-bit sizes: no overflow at the largest call
    assert L.exl3_lora_workspace_size(1 << 26, 65536, 128, 1024) >= (1 << 26) * 128 * 4


def test_binding_refuses_wrong_shapes_and_layouts():
    x = torch.zeros(4, 64, dtype=torch.float16)
    a, b = torch.zeros(2, 8, 64, dtype=torch.float16), torch.zeros(2, 32, 8, dtype=torch.float16)
    ids = torch.zeros(4, dtype=torch.int32)
    E = exl3.Exl3Error
    for bad in (dict(x=x.t()), dict(a=a[:, :, :32]), dict(b=b.transpose(1, 2)),
                dict(a=a.to(torch.bfloat16)), dict(ids=ids[:3]), dict(scale=torch.ones(3)),
                dict(ranks=torch.ones(2)), dict(base=torch.zeros(4, 16)),
                dict(out=torch.zeros(3, 32)), dict(base=torch.zeros(32, 4).t())):
        with pytest.raises(E):
            exl3.exl3_lora(**{**dict(x=x, a=a, b=b, ids=ids), **bad})
    l = torch.zeros(4, 16)
    for bad in (dict(logits=l.t()[:, ::2]), dict(scoring="relu"), dict(bias=torch.zeros(15)),
                dict(row_mask=torch.zeros(4)), dict(row_mask=torch.zeros(3, dtype=torch.bool)),
                dict(ids=torch.zeros(4, 3, dtype=torch.int32)), dict(w=torch.zeros(2, 4).t())):
        with pytest.raises(E):
            exl3.exl3_route_topk(**{**dict(logits=l, topk=2), **bad})
    with pytest.raises(E):
        exl3.exl3_balance_loss(l, torch.zeros(3, 2, dtype=torch.int32))
    with pytest.raises(E):
        exl3.exl3_route_backward(l, torch.zeros(4, 2, dtype=torch.int32), dw=torch.zeros(4, 3))
