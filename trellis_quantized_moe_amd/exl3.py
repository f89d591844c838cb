"""ctypes binding of libexl3moe.so (C ABI in include/exl3moe.h).

Argument marshalling only: every step of the layer runs in the HIP library.
torch provides device memory and the current stream. If the library is not
built, every call raises; there is no fallback path.
"""

import ctypes
import functools
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libexl3moe.so")

F16, BF16, F32, I32, I64 = 1, 2, 3, 4, 5
_DT = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32,
       torch.int32: I32, torch.int64: I64}
_OUT = {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32}


def _dt(t):
    """Library dtype code of a tensor; 0 (rejected by the library) if it has none."""
    return _DT.get(t.dtype, 0)


class Exl3Error(RuntimeError):
    pass


class ProjC(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("num_stages", ctypes.c_int32),
                ("trellis", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("bits", ctypes.c_void_p), ("suh", ctypes.c_void_p),
                ("svh", ctypes.c_void_p), ("chscale", ctypes.c_void_p)]


class MetaC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("expert_count", "expert_offset", "pair_of_pos", "weight_of_pos",
                 "pos_of_pair", "num_active", "status")]


class ProfileC(ctypes.Structure):
    _fields_ = [("events", ctypes.POINTER(ctypes.c_void_p)),
                ("kernel_ids", ctypes.POINTER(ctypes.c_int32)),
                ("cap", ctypes.c_int32), ("n", ctypes.c_int32)]


class RouterC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_experts", "topk", "scoring", "renorm")] + [
        ("scale", ctypes.c_float), ("bias", ctypes.c_void_p)]


class BalanceC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("count", "tokens", "prob", "loss")]


class LoraC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("in_features", "out_features", "rank", "num_adapters")] + [
        (n, ctypes.c_void_p) for n in ("a", "b", "scale", "ranks")]


class W4C(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("in_features", "out_features", "num_experts", "group_size")] + [
        (n, ctypes.c_void_p) for n in ("q", "scale", "zero")] + [("scale_dtype", ctypes.c_int32)]


class LayoutC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("ctrl", "meta", "expert_of_pos", "plan", "xt", "at", "d", "yacc",
                 "total")] + [("passes", ctypes.c_int32), ("plan_slots", ctypes.c_int32),
                              ("plan_group", ctypes.c_int32)]


_lib = None
_i32, _sz, _vp = ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
_i64, _f32 = ctypes.c_int64, ctypes.c_float
_PP = ctypes.POINTER(ProfileC)
_SIGS = {
    "exl3_abi_version": (_i32, []),
    "exl3_status_string": (ctypes.c_char_p, [_i32]),
    "exl3_route_pack": (_i32, [_vp, _i32, _vp, _i32, _i32, _i32, _i32,
                               ctypes.POINTER(MetaC), _vp, _PP]),
    "exl3_linear_workspace_size": (_sz, [_i32, _i32, _i32]),
    "exl3_linear": (_i32, [_vp, _i32, _i32, ctypes.POINTER(ProjC), _vp, _i32, _vp, _sz,
                           _vp, _PP]),
    "exl3_moe_workspace_size": (_sz, [_i32] * 6),
    "exl3_moe_forward": (_i32, [_vp, _i32, _i32, _vp, _i32, _vp, _i32, _i32,
                                ctypes.POINTER(ProjC), ctypes.POINTER(ProjC),
                                ctypes.POINTER(ProjC), _vp, _i32, _i32, _i32, _vp, _sz,
                                _vp, _PP]),
    "exl3_moe_forward_static": (_i32, [_vp, _i32, _i32, _vp, _i32, _vp, _i32, _i32,
                                       ctypes.POINTER(ProjC), ctypes.POINTER(ProjC),
                                       ctypes.POINTER(ProjC), _vp, _i32, _i32, _i32, _vp,
                                       _PP]),
    "exl3_moe_additive": (_i32, [_vp, _i32, _i32, _i32, ctypes.POINTER(MetaC),
                                 ctypes.POINTER(ProjC), ctypes.POINTER(ProjC),
                                 ctypes.POINTER(ProjC), _vp, _i32, _i32, _i32, _vp, _sz,
                                 _vp, _PP]),
    "exl3_moe_layout": (_i32, [_i32] * 6 + [ctypes.POINTER(LayoutC)]),
    "exl3_route_topk": (_i32, [ctypes.POINTER(RouterC), _vp, _i32, _i64, _i32, _vp, _vp, _i32,
                               _vp, _i32, _vp, _PP]),
    "exl3_balance_workspace_size": (_sz, [_i32, _i32]),
    "exl3_balance_loss": (_i32, [ctypes.POINTER(RouterC), _vp, _i32, _i64, _i32, _vp, _i32, _f32,
                                 ctypes.POINTER(BalanceC), _vp, _sz, _vp, _PP]),
    "exl3_route_backward": (_i32, [ctypes.POINTER(RouterC), _vp, _i32, _i64, _i32, _vp, _i32, _vp,
                                   _i32, ctypes.POINTER(BalanceC), _f32, _vp, _vp, _i32, _i64,
                                   _vp, _PP]),
    "exl3_lora_workspace_size": (_sz, [_i32] * 4),
    "exl3_lora": (_i32, [ctypes.POINTER(LoraC), _vp, _i32, _i64, _i32, _vp, _i32, _vp, _i32, _i64,
                         _vp, _i32, _i64, _vp, _sz, _vp, _PP]),
    "exl3_permute": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _i64, _vp, _PP]),
    "exl3_unpermute": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _i32, _i64,
                              _vp, _PP]),
    "exl3_unpermute_backward": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _i32, _i64,
                                       _vp, _i32, _vp, _i64, _vp, _i32, _vp, _PP]),
    "exl3_w4_linear": (_i32, [ctypes.POINTER(W4C), _vp, _i32, _i64, _i32, _vp, _vp, _i32, _i64,
                              _vp, _PP]),
    "exl3_decode_tiles": (_i32, [_vp, _i32, _i32, _vp, _vp, _PP]),
    "exl3_events_create": (_i32, [_i32, ctypes.POINTER(ctypes.c_void_p)]),
    "exl3_events_destroy": (_i32, [_i32, ctypes.POINTER(ctypes.c_void_p)]),
    "exl3_profile_read": (_i32, [_PP, ctypes.POINTER(ctypes.c_float)]),
}
KERNEL_NAMES = {1: "route_pack", 2: "rotate", 3: "gemm_gateup", 4: "gemm_down",
                5: "combine", 6: "gemm_linear", 7: "decode_tiles", 8: "gemm_experts",
                9: "route_topk", 10: "balance", 11: "balance_sum", 12: "route_backward",
                13: "lora_a", 14: "lora_b", 15: "lora", 16: "permute", 17: "unpermute",
                18: "unpermute_backward", 19: "w4"}


def lib():
    """Load libexl3moe.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise Exl3Error("%s is missing: build it with __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status):
    if status != 0:
        raise Exl3Error("exl3 status %d: %s" % (status, lib().exl3_status_string(status).decode()))


def _stream():
    # the current stream's handle without building a Stream object (0.3 us
    # instead of 2.8: a third of a small call's time on the host)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _p(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def abi_version():
    return lib().exl3_abi_version()


class DeviceProj:
    """A projection's tables and tensors resident on the GPU.

    ``proj`` is any object with in_features, out_features, num_experts,
    words[t][e] (flat uint16 numpy or None), scale, bits, suh, svh, chscale
    (e.g. ``synth.Proj``). All trellis tensors live in one device buffer,
    each 256-byte aligned; the int64 pointer table addresses into it.
    """

    def __init__(self, proj, device="cuda", words_fn=None):
        S = len(proj.words)
        E = proj.num_experts
        self.in_features, self.out_features = proj.in_features, proj.out_features
        self.num_experts, self.num_stages = E, S
        offs = np.zeros((S, E), dtype=np.int64)
        total = 0
        sizes = {}
        for t in range(S):
            for e in range(E):
                w = proj.words[t][e]
                if w is None:
                    offs[t, e] = -1
                    continue
                n = (proj.in_features // 16) * (proj.out_features // 16) * 16 * int(proj.bits[t][e])
                sizes[(t, e)] = n
                offs[t, e] = total
                total += (2 * n + 255) // 256 * 256
        self.buffer = torch.empty(max(total, 256), dtype=torch.uint8, device=device)
        base = self.buffer.data_ptr()
        for (t, e), n in sizes.items():
            w = proj.words[t][e]
            if words_fn is not None and not isinstance(w, np.ndarray):
                w = words_fn(proj, t, e)
            arr = torch.from_numpy(np.ascontiguousarray(w).view(np.uint8))
            o = int(offs[t, e])
            self.buffer[o:o + 2 * n].copy_(arr, non_blocking=False)
        ptrs = np.where(offs >= 0, offs + base, 0).astype(np.int64)
        self.trellis = torch.from_numpy(ptrs).to(device)
        self.scale = torch.from_numpy(np.asarray(proj.scale, np.float32).copy()).to(device)
        self.bits = torch.from_numpy(np.asarray(proj.bits, np.int32).copy()).to(device)
        self.suh = torch.from_numpy(np.asarray(proj.suh, np.float16).copy()).to(device)
        self.svh = torch.from_numpy(np.asarray(proj.svh, np.float16).copy()).to(device)
        self.chscale = torch.from_numpy(np.asarray(proj.chscale, np.float16).copy()).to(device)
        self.offsets = offs

    def cstruct(self):
        return ProjC(self.in_features, self.out_features, self.num_experts,
                     self.num_stages, self.trellis.data_ptr(), self.scale.data_ptr(),
                     self.bits.data_ptr(), self.suh.data_ptr(), self.svh.data_ptr(),
                     self.chscale.data_ptr())

    def trellis_bytes(self, t, e):
        """Bytes of the (stage, expert) trellis, 0 if absent."""
        if self.offsets[t, e] < 0:
            return 0
        return (self.in_features // 16) * (self.out_features // 16) * 32 * int(
            self.bits[t, e].item())


def alloc_meta(rows, topk, num_experts, device="cuda"):
    P = rows * topk
    i32 = dict(dtype=torch.int32, device=device)
    return {
        "expert_count": torch.empty(num_experts, **i32),
        "expert_offset": torch.empty(num_experts + 1, **i32),
        "pair_of_pos": torch.empty(max(P, 1), **i32),
        "weight_of_pos": torch.empty(max(P, 1), dtype=torch.float32, device=device),
        "pos_of_pair": torch.empty(max(P, 1), **i32),
        "num_active": torch.empty(4, **i32),
        "status": torch.empty(4, **i32),
    }


def _meta_c(m):
    return MetaC(*[m[n].data_ptr() for n in
                   ("expert_count", "expert_offset", "pair_of_pos", "weight_of_pos",
                    "pos_of_pair", "num_active", "status")])


def exl3_route_pack(ids, w, num_experts, meta=None):
    rows, topk = ids.shape
    meta = meta or alloc_meta(rows, topk, num_experts, ids.device)
    mc = _meta_c(meta)
    _check(lib().exl3_route_pack(_p(ids), _DT[ids.dtype], _p(w), _DT[w.dtype], rows, topk,
                                 num_experts, ctypes.byref(mc), _stream(), _prof()))
    return meta


def linear_workspace_size(rows, in_f, out_f):
    return lib().exl3_linear_workspace_size(rows, in_f, out_f)


def exl3_linear(x, proj, out_dtype=torch.float32, out=None, ws=None):
    rows = x.shape[0]
    out = out if out is not None else torch.empty(rows, proj.out_features, dtype=out_dtype,
                                                  device=x.device)
    need = linear_workspace_size(rows, proj.in_features, proj.out_features)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    pc = proj.cstruct()
    _check(lib().exl3_linear(_p(x), _dt(x), rows, ctypes.byref(pc), _p(out), _DT[out.dtype],
                             _p(ws), ws.numel(), _stream(), _prof()))
    return out


def moe_layout(rows, topk, num_experts, hidden, intermediate, capacity):
    lay = LayoutC()
    _check(lib().exl3_moe_layout(rows, topk, num_experts, hidden, intermediate, capacity,
                                 ctypes.byref(lay)))
    return lay


def moe_workspace_size(rows, topk, num_experts, hidden, intermediate, capacity):
    return lib().exl3_moe_workspace_size(rows, topk, num_experts, hidden, intermediate,
                                         capacity)


def exl3_moe_forward(x, ids, w, gate, up, down, capacity, out_dtype=torch.float32,
                     out=None, ws=None, num_active_hint=-1):
    rows, topk = ids.shape
    out = out if out is not None else torch.empty(rows, down.out_features, dtype=out_dtype,
                                                  device=x.device)
    need = moe_workspace_size(rows, topk, gate.num_experts, gate.in_features,
                              gate.out_features, capacity)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    g, u, d = gate.cstruct(), up.cstruct(), down.cstruct()
    _check(lib().exl3_moe_forward(_p(x), _dt(x), rows, _p(ids), _DT[ids.dtype], _p(w),
                                  _DT[w.dtype], topk, ctypes.byref(g), ctypes.byref(u),
                                  ctypes.byref(d), _p(out), _DT[out.dtype], capacity,
                                  num_active_hint,
                                  _p(ws), ws.numel(), _stream(), _prof()))
    return out


def exl3_moe_forward_static(x, ids, w, gate, up, down, capacity, out_dtype=torch.float32,
                            out=None, num_active_hint=-1):
    """exl3_moe_forward on the library's static scratch (no workspace)."""
    rows, topk = ids.shape
    out = out if out is not None else torch.empty(rows, down.out_features, dtype=out_dtype,
                                                  device=x.device)
    g, u, d = gate.cstruct(), up.cstruct(), down.cstruct()
    _check(lib().exl3_moe_forward_static(_p(x), _dt(x), rows, _p(ids), _DT[ids.dtype], _p(w),
                                         _DT[w.dtype], topk, ctypes.byref(g), ctypes.byref(u),
                                         ctypes.byref(d), _p(out), _DT[out.dtype], capacity,
                                         num_active_hint, _stream(), _prof()))
    return out


STATIC_SCRATCH_BYTES = 32 << 20


def exl3_moe_additive(x, topk, meta, gate, up, down, capacity, out_dtype=torch.float32,
                      out=None, ws=None, num_active_hint=-1):
    rows = x.shape[0]
    out = out if out is not None else torch.empty(rows, down.out_features, dtype=out_dtype,
                                                  device=x.device)
    need = moe_workspace_size(rows, topk, gate.num_experts, gate.in_features,
                              gate.out_features, capacity)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    g, u, d = gate.cstruct(), up.cstruct(), down.cstruct()
    mc = _meta_c(meta)
    _check(lib().exl3_moe_additive(_p(x), _dt(x), rows, topk, ctypes.byref(mc),
                                   ctypes.byref(g), ctypes.byref(u), ctypes.byref(d), _p(out),
                                   _DT[out.dtype], capacity, num_active_hint, _p(ws), ws.numel(), _stream(),
                                   _prof()))
    return out


# ------------------------------------------------------- router operators
SCORING = {"softmax": 0, "sigmoid": 1}


def _refuse(what, *args):
    """Shapes and layouts that the C ABI, given bare pointers, cannot check."""
    raise Exl3Error(what % args)


_MAX = 0x7fffffff  # sizes of the C ABI: ctypes would cut a larger one off to 32 bits


def _too_large(*sizes):
    _refuse("a size of %d is out of range", max(sizes))


def _matrix(t, rows, cols, name):
    """Row distance of a [rows][cols] tensor whose rows are contiguous."""
    if t.shape != (rows, cols):
        _refuse("%s must be [%d, %d], got %s", name, rows, cols, list(t.shape))
    ld, step = t.stride()
    if step != 1 and cols != 1:
        _refuse("%s must have contiguous rows", name)
    return ld if rows > 1 else cols


def _vector(t, n, dtype, name):
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        _refuse("%s must be %d contiguous values of %s", name, n, dtype)
    return t.data_ptr()


def _workspace(ws, need, device):
    """The caller's workspace, or a new one: its bytes lie side by side."""
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if not ws.is_contiguous():
        _refuse("ws must be contiguous")
    return ws


def _pairs(t, rows, topk, name):
    if t.shape != (rows, topk) or not t.is_contiguous():
        _refuse("%s must be contiguous [%d, %d], got %s", name, rows, topk, list(t.shape))
    return t.data_ptr()


def _router_c(E, topk, scoring, renorm=True, scale=1.0, bias=None):
    if scoring not in SCORING:
        _refuse("scoring must be 'softmax' or 'sigmoid', got %r", scoring)
    if topk > _MAX:
        _too_large(topk)
    return RouterC(E, topk, SCORING[scoring], 1 if renorm else 0, scale, bias)


def _logits(logits):
    if logits.dim() != 2:
        _refuse("logits must be [rows, experts], got %s", list(logits.shape))
    rows, E = logits.shape
    if rows > _MAX or E > _MAX:
        _too_large(rows, E)
    return rows, E, _matrix(logits, rows, E, "logits")


def exl3_route_topk(logits, topk, scoring="softmax", renorm=True, scale=1.0, bias=None,
                    row_mask=None, ids_dtype=torch.int32, w_dtype=torch.float32, ids=None, w=None):
    """Router logits [rows, experts] -> (ids, w), both [rows, topk]: the topk
    best experts of every row and their route weights, as exl3_moe_forward
    takes them. ``bias`` (fp32 [experts]) moves the choice only; rows whose
    ``row_mask`` (bool or uint8 [rows]) is 0 get ID -1 and weight 0. The results
    are not part of autograd's graph: a program that trains the router calls
    exl3_route_backward itself."""
    rows, E, ld = _logits(logits)
    if bias is not None:
        bias = _vector(bias, E, torch.float32, "bias")
    mask = None
    if row_mask is not None:
        if row_mask.dtype is not torch.bool and row_mask.dtype is not torch.uint8:
            _refuse("row_mask must be bool or uint8, got %s", row_mask.dtype)
        mask = _vector(row_mask, rows, row_mask.dtype, "row_mask")
    if ids is None:
        ids = torch.empty(rows, topk, dtype=ids_dtype, device=logits.device)
    if w is None:
        w = torch.empty(rows, topk, dtype=w_dtype, device=logits.device)
    rc = _router_c(E, topk, scoring, renorm, scale, bias)
    _check(lib().exl3_route_topk(ctypes.byref(rc), logits.data_ptr(), _dt(logits), ld, rows, mask,
                                 _pairs(ids, rows, topk, "ids"), _dt(ids),
                                 _pairs(w, rows, topk, "w"), _dt(w), _stream(), _prof()))
    return ids, w


def alloc_balance(num_experts, device="cuda"):
    return {
        "count": torch.empty(num_experts, dtype=torch.int32, device=device),
        "tokens": torch.empty(1, dtype=torch.int32, device=device),
        "prob": torch.empty(num_experts, dtype=torch.float32, device=device),
        "loss": torch.empty(1, dtype=torch.float32, device=device),
    }


@functools.lru_cache(maxsize=1024)
def balance_workspace_size(rows, num_experts):
    if rows > _MAX or num_experts > _MAX:
        _too_large(rows, num_experts)
    return lib().exl3_balance_workspace_size(rows, num_experts)


def _ids_of(ids, rows):
    """topk and address of routed IDs [rows, topk]."""
    if ids.dim() != 2:
        _refuse("ids must be [rows, topk], got %s", list(ids.shape))
    return ids.shape[1], _pairs(ids, rows, ids.shape[1], "ids")


def exl3_balance_loss(logits, ids, scoring="softmax", coef=1.0, balance=None, ws=None):
    """Balance loss of a routing and its per-expert statistics: a dict with
    "loss" [1], "count" [experts], "prob" [experts] and "tokens" [1]. Not part
    of autograd's graph; exl3_route_backward gives the gradient."""
    rows, E, ld = _logits(logits)
    topk, idp = _ids_of(ids, rows)
    if balance is None:
        balance = alloc_balance(E, logits.device)
    ws = _workspace(ws, balance_workspace_size(rows, E), logits.device)
    rc = _router_c(E, topk, scoring)
    bc = BalanceC(_vector(balance["count"], E, torch.int32, "count"),
                  _vector(balance["tokens"], 1, torch.int32, "tokens"),
                  _vector(balance["prob"], E, torch.float32, "prob"),
                  _vector(balance["loss"], 1, torch.float32, "loss"))
    _check(lib().exl3_balance_loss(ctypes.byref(rc), logits.data_ptr(), _dt(logits), ld, rows, idp,
                                   _dt(ids), coef, ctypes.byref(bc), ws.data_ptr(), ws.numel(),
                                   _stream(), _prof()))
    return balance


def exl3_route_backward(logits, ids, dw=None, scoring="softmax", renorm=True, scale=1.0,
                        balance=None, coef=1.0, dloss=None, dlogits_dtype=None, dlogits=None):
    """Gradient with respect to the router's logits: of the route weights
    (``dw`` [rows, topk]), of the balance loss (``balance`` as
    exl3_balance_loss returned it, with ``dloss`` fp32 [1] or None for 1), or
    of both together. ``dw`` is the caller's: exl3_moe_forward has no backward
    pass."""
    rows, E, ld = _logits(logits)
    topk, idp = _ids_of(ids, rows)
    dwp, dwt = None, 0
    if dw is not None:
        dwp, dwt = _pairs(dw, rows, topk, "dw"), _dt(dw)
    if dlogits is None:
        dlogits = torch.empty(rows, E, dtype=dlogits_dtype or logits.dtype, device=logits.device)
    bc = None
    if balance is not None:
        bc = ctypes.byref(BalanceC(_vector(balance["count"], E, torch.int32, "count"),
                                   _vector(balance["tokens"], 1, torch.int32, "tokens"),
                                   None, None))
    if dloss is not None:
        dloss = _vector(dloss, 1, torch.float32, "dloss")
    rc = _router_c(E, topk, scoring, renorm, scale)
    _check(lib().exl3_route_backward(ctypes.byref(rc), logits.data_ptr(), _dt(logits), ld, rows,
                                     idp, _dt(ids), dwp, dwt, bc, coef, dloss, dlogits.data_ptr(),
                                     _dt(dlogits), _matrix(dlogits, rows, E, "dlogits"),
                                     _stream(), _prof()))
    return dlogits


@functools.lru_cache(maxsize=1024)
def lora_workspace_size(rows, in_f, rank, num_adapters):
    if max(rows, in_f, rank, num_adapters) > _MAX:
        _too_large(rows, in_f, rank, num_adapters)
    return lib().exl3_lora_workspace_size(rows, in_f, rank, num_adapters)


def exl3_lora(x, a, b, ids, scale=None, ranks=None, base=None, out_dtype=None, out=None, ws=None):
    """Low-rank adapters beside a shared projection: row t gets
    ``base[t] + scale[i] * (x[t] @ a[i].T) @ b[i].T`` with i = ids[t], or
    ``base[t]`` (zeros without a base) where ids[t] names no adapter.

    x [rows, in], a [adapters, rank, in] and b [adapters, out, rank] share one
    16-bit dtype; ``scale`` (fp32) and ``ranks`` (int32, the ranks in use) hold
    one value per adapter. ``base`` and ``out`` [rows, out] may be column
    slices of wider tensors; ``out=base`` adds in place. Without ``out`` the
    result has ``out_dtype``, by default that of ``base`` or else of ``x``. The
    result is not part of autograd's graph."""
    if x.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        _refuse("x must have two dimensions, a and b three")
    rows, K = x.shape
    n, N, R = b.shape
    if rows > _MAX or K > _MAX or n > _MAX or N > _MAX or R > _MAX:
        _too_large(rows, K, n, N, R)
    if a.shape != (n, R, K):
        _refuse("a must be [adapters, rank, in] and b [adapters, out, rank], got %s and %s",
                list(a.shape), list(b.shape))
    if a.dtype is not x.dtype or b.dtype is not x.dtype:
        _refuse("x, a and b must share one dtype")
    if not (a.is_contiguous() and b.is_contiguous()):
        _refuse("a and b must be contiguous")
    if ids.shape != (rows,) or not ids.is_contiguous():
        _refuse("ids must be contiguous [%d]", rows)
    if scale is not None:
        scale = _vector(scale, n, torch.float32, "scale")
    if ranks is not None:
        ranks = _vector(ranks, n, torch.int32, "ranks")
    basep, baset, ldb = None, 0, 0
    if base is not None:
        basep, baset, ldb = base.data_ptr(), _dt(base), _matrix(base, rows, N, "base")
    if out is None:
        out = torch.empty(rows, N, device=x.device,
                          dtype=out_dtype or (base.dtype if base is not None else x.dtype))
    ws = _workspace(ws, max(lora_workspace_size(rows, K, R, n), 256), x.device)
    lc = LoraC(K, N, R, n, a.data_ptr(), b.data_ptr(), scale, ranks)
    _check(lib().exl3_lora(ctypes.byref(lc), x.data_ptr(), _dt(x), _matrix(x, rows, K, "x"), rows,
                           ids.data_ptr(), _dt(ids), basep, baset, ldb, out.data_ptr(), _dt(out),
                           _matrix(out, rows, N, "out"), ws.data_ptr(), ws.numel(), _stream(),
                           _prof()))
    return out


# ------------------------------------- rows to experts and their products
def _pos(meta, rows, topk):
    """Address of the packed positions of rows * topk choices."""
    if topk < 1 or rows * topk > _MAX:
        _refuse("%d choices of %d rows are out of range", topk, rows)
    pos = meta["pos_of_pair"]
    # alloc_meta's buffers have one element where a batch has none
    return _vector(pos, rows * topk or min(pos.numel(), 1), torch.int32, "pos_of_pair")


def _packed(t, topk, name):
    """Rows and features of a packed tensor [rows * topk, features]."""
    if t.dim() != 2 or topk < 1 or t.shape[0] % topk:
        _refuse("%s must be [rows * %d, features], got %s", name, topk, list(t.shape))
    return t.shape[0] // topk, t.shape[1]


def exl3_permute(x, meta, topk, out=None):
    """Rows x [rows, features] to their experts: out [rows * topk, features]
    holds x[t] at the packed position of every choice of row t. ``meta`` is
    exl3_route_pack's (its "pos_of_pair" is read). Packed rows past the last
    kept pair keep what ``out`` held (without ``out``: anything). The gradient
    with respect to x is exl3_unpermute of the gradient of out, without w."""
    if x.dim() != 2:
        _refuse("x must be [rows, features], got %s", list(x.shape))
    rows, H = x.shape
    if rows > _MAX or H > _MAX:
        _too_large(rows, H)
    pos = _pos(meta, rows, topk)
    if out is None:
        out = torch.empty(rows * topk, H, dtype=x.dtype, device=x.device)
    elif out.dtype is not x.dtype:
        _refuse("out must have the dtype of x, %s, got %s", x.dtype, out.dtype)
    _check(lib().exl3_permute(x.data_ptr(), _dt(x), _matrix(x, rows, H, "x"), rows, topk, H, pos,
                              out.data_ptr(), _matrix(out, rows * topk, H, "out"), _stream(),
                              _prof()))
    return out


def exl3_unpermute(y, meta, topk, w=None, out_dtype=None, out=None):
    """Experts' results y [rows * topk, features] back to their rows: out[t] is
    the sum of y at the packed positions of row t's choices, each times its
    route weight w [rows, topk] (without w: 1). Dropped choices take no part.
    The result is not part of autograd's graph; exl3_unpermute_backward gives
    the gradient."""
    rows, H = _packed(y, topk, "y")
    if y.shape[0] > _MAX or H > _MAX:
        _too_large(y.shape[0], H)
    pos = _pos(meta, rows, topk)
    wp, wt = None, 0
    if w is not None:
        wp, wt = _pairs(w, rows, topk, "w"), _dt(w)
    if out is None:
        out = torch.empty(rows, H, dtype=out_dtype or y.dtype, device=y.device)
    _check(lib().exl3_unpermute(y.data_ptr(), _dt(y), _matrix(y, rows * topk, H, "y"), rows, topk,
                                H, pos, wp, wt, out.data_ptr(), _dt(out),
                                _matrix(out, rows, H, "out"), _stream(), _prof()))
    return out


def exl3_unpermute_backward(dout, meta, topk, y=None, w=None, dy_dtype=None, dw_dtype=None, dy=None,
                            dw=None):
    """Gradient of exl3_unpermute: (dy, dw) from dout [rows, features], the
    gradient of its result. dy [rows * topk, features] has the dtype of ``y``
    (without y: ``dy_dtype``, by default that of dout); packed rows past the
    last kept pair keep what ``dy`` held. dw [rows, topk] is what
    exl3_route_backward takes; it needs ``y`` and is None without it."""
    if dout.dim() != 2:
        _refuse("dout must be [rows, features], got %s", list(dout.shape))
    rows, H = dout.shape
    if rows > _MAX or H > _MAX:
        _too_large(rows, H)
    pos = _pos(meta, rows, topk)
    yp, ldy, wp, wt, dwp, dwt = None, 0, None, 0, None, 0
    if w is not None:
        wp, wt = _pairs(w, rows, topk, "w"), _dt(w)
    if dy is None:
        dy = torch.empty(rows * topk, H, device=dout.device,
                         dtype=y.dtype if y is not None else dy_dtype or dout.dtype)
    if y is not None:
        if y.dtype is not dy.dtype:
            _refuse("dy must have the dtype of y, %s, got %s", y.dtype, dy.dtype)
        yp, ldy = y.data_ptr(), _matrix(y, rows * topk, H, "y")
        if dw is None:
            dw = torch.empty(rows, topk, device=dout.device,
                             dtype=dw_dtype or (w.dtype if w is not None else torch.float32))
        dwp, dwt = _pairs(dw, rows, topk, "dw"), _dt(dw)
    elif dw is not None:
        _refuse("dw needs y")
    _check(lib().exl3_unpermute_backward(dout.data_ptr(), _dt(dout),
                                         _matrix(dout, rows, H, "dout"), rows, topk, H, pos, yp,
                                         _dt(dy), ldy, wp, wt, dy.data_ptr(),
                                         _matrix(dy, rows * topk, H, "dy"), dwp, dwt, _stream(),
                                         _prof()))
    return dy, dw


class DeviceW4:
    """4-bit weights of a projection, of one expert or several, laid out for
    exl3_w4_linear on the device that they are on.

    ``q`` uint8 [experts, out, in / 2] (or [out, in / 2]) holds two weights a
    byte, the even input in the lower four bits; ``scale`` fp16 or bf16
    [experts, out, in / group] and ``zero`` (uint8 of 0..15, the same shape; None:
    8) belong to groups of 32, 64 or 128 inputs: weight = scale * (q - zero).
    Outputs are a multiple of 8, inputs and outputs at most 65536, experts at
    most 1024. The tensors given are not kept."""

    @torch.no_grad()
    def __init__(self, q, scale, zero=None):
        if q.dim() == 2:
            q, scale = q[None], scale[None]
            zero = None if zero is None else zero[None]
        if q.dim() != 3 or q.dtype != torch.uint8 or 0 in q.shape:
            _refuse("q must be uint8 [experts, out, in / 2], got %s of %s", list(q.shape), q.dtype)
        E, N, K = q.shape[0], q.shape[1], 2 * q.shape[2]
        if scale.dim() != 3 or scale.shape[:2] != (E, N) or scale.dtype not in (torch.float16,
                                                                               torch.bfloat16):
            _refuse("scale must be fp16 or bf16 [%d, %d, groups], got %s of %s", E, N,
                    list(scale.shape), scale.dtype)
        group = next((g for g in (32, 64, 128) if g * scale.shape[2] == K), 0)
        if not group:
            _refuse("%d inputs in %d groups: groups must have 32, 64 or 128", K, scale.shape[2])
        if zero is not None:
            if zero.shape != scale.shape or zero.dtype != torch.uint8:
                _refuse("zero must be uint8 %s, got %s of %s", list(scale.shape),
                        list(zero.shape), zero.dtype)
            if int(zero.max()) > 15:
                _refuse("zero has values above 15")
        if max(E, N, K) > _MAX:
            _too_large(E, N, K)
        # the limits of the products: a call without rows checks no more
        none = W4C(K, N, E, group, None, None, None, _dt(scale))
        _check(lib().exl3_w4_linear(ctypes.byref(none), None, F16, K, 0, None, None, F16, N, None,
                                    None))
        self.in_features, self.out_features = K, N
        self.num_experts, self.group_size = E, group
        NT, KT, NG = (N + 15) // 16, (K + 127) // 128, 128 // group
        self.q = torch.empty(E, NT, KT, 64, 16, dtype=torch.uint8, device=q.device)
        self.scale = torch.empty(E, NT, KT, 16, NG, dtype=scale.dtype, device=q.device)
        self.zero = None if zero is None else torch.empty_like(self.scale, dtype=torch.uint8)

        def padded(t, cols):  # outputs and columns that the tiles have and t lacks: 0
            return torch.nn.functional.pad(t, (0, cols - t.shape[2], 0, 16 * NT - N))

        step = max(1, (1 << 27) // (N * K))  # experts at a time: little extra memory
        for e in range(0, E, step):
            w = q[e:e + step].reshape(-1)
            if w.storage_offset() % 4:
                w = w.clone()
            w = w.view(torch.int32).view(-1, N, K // 8)  # inputs 0 .. 7 from bit 0 on
            even, odd = w & 0x0f0f0f0f, (w >> 4) & 0x0f0f0f0f
            for sh, mask in ((4, 0x00ff00ff), (8, 0x0000ffff)):
                even, odd = (even | even >> sh) & mask, (odd | odd >> sh) & mask
            w = padded(even | odd << 16, 16 * KT).reshape(-1, NT, 16, KT, 4, 4)
            # output, tile, word, lane group -> tile, lane group, output, word
            w = w.permute(0, 1, 3, 5, 2, 4).contiguous()
            self.q[e:e + step] = w.view(torch.uint8).reshape(-1, NT, KT, 64, 16)
            for to, t in ((self.scale, scale), (self.zero, zero)):
                if t is not None:
                    t = padded(t[e:e + step], KT * NG).reshape(-1, NT, 16, KT, NG)
                    to[e:e + step] = t.transpose(2, 3)
        self._c = W4C(K, N, E, group, self.q.data_ptr(), self.scale.data_ptr(),
                      0 if zero is None else self.zero.data_ptr(), _dt(scale))

    def cstruct(self):
        return self._c


def exl3_w4_linear(x, weight, expert_offset=None, out_dtype=None, out=None):
    """x [rows, in] times the transposed 4-bit weights (a DeviceW4): packed rows
    with their experts' weights, where ``expert_offset`` is exl3_route_pack's
    "expert_offset", or all rows with a single projection's. x is fp16 or bf16;
    x and ``out`` [rows, out] may be column slices of wider tensors. Without
    ``out`` the result has ``out_dtype``, by default that of x; rows past the
    last expert's keep what ``out`` held (without ``out``: anything). A group's
    sum is formed before its scale, in fp32: bf16 x from 2^117 on may overflow
    it. The result is not part of autograd's graph."""
    if x.dim() != 2:
        _refuse("x must be [rows, in], got %s", list(x.shape))
    rows, N = x.shape[0], weight.out_features
    if rows > _MAX:
        _too_large(rows)
    if expert_offset is not None:
        expert_offset = _vector(expert_offset, weight.num_experts + 1, torch.int32,
                                "expert_offset")
    if out is None:
        out = torch.empty(rows, N, dtype=out_dtype or x.dtype, device=x.device)
    _check(lib().exl3_w4_linear(ctypes.byref(weight.cstruct()), x.data_ptr(), _dt(x),
                                _matrix(x, rows, weight.in_features, "x"), rows, expert_offset,
                                out.data_ptr(), _dt(out), _matrix(out, rows, N, "out"), _stream(),
                                _prof()))
    return out


def exl3_decode_tiles(words, K):
    """words: uint16-bit tensor (int16 view) [ntiles * 16K] -> fp16 [ntiles][16][16]."""
    ntiles = words.numel() // (16 * K)
    out = torch.empty(ntiles, 16, 16, dtype=torch.float16, device=words.device)
    _check(lib().exl3_decode_tiles(_p(words), ntiles, K, _p(out), _stream(), _prof()))
    return out


def unpermute_rotated(t):
    """Undo the in-group storage order of rotated vectors read from the
    workspace (slot p of each 16-group holds entry kSigma[p])."""
    sigma = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7, 8, 12, 9, 13, 10, 14, 11, 15],
                         device=t.device)
    shape = t.shape
    g = t.reshape(*shape[:-1], shape[-1] // 16, 16)
    out = torch.empty_like(g)
    out[..., sigma] = g
    return out.reshape(shape)


_active_profile = None


def _prof():
    """The caller-owned timing record of the enclosing ``Profile`` block, or None."""
    return ctypes.byref(_active_profile.c) if _active_profile is not None else None


class Profile:
    """Per-launch kernel timing: ``with Profile(n) as p: ...`` then
    ``p.records`` = [(name, ms), ...]. The events are created on entry and
    destroyed on exit (outside the calls being timed); inside the block every
    call of this module passes the record to the library, which brackets each
    of its launches with the next event pair."""

    def __init__(self, max_launches=4096):
        self.max = max_launches
        self.records = []

    def __enter__(self):
        global _active_profile
        if _active_profile is not None:
            raise Exl3Error("Profile blocks do not nest")
        self._events = (ctypes.c_void_p * (2 * self.max))()
        self._ids = (ctypes.c_int32 * self.max)()
        _check(lib().exl3_events_create(2 * self.max, self._events))
        self.c = ProfileC(self._events, self._ids, self.max, 0)
        _active_profile = self
        return self

    def __exit__(self, *exc):
        global _active_profile
        _active_profile = None
        ms = (ctypes.c_float * self.max)()
        try:
            _check(lib().exl3_profile_read(ctypes.byref(self.c), ms))
            self.records = [(KERNEL_NAMES.get(self._ids[i], str(self._ids[i])), float(ms[i]))
                            for i in range(self.c.n)]
        finally:
            lib().exl3_events_destroy(2 * self.max, self._events)
        return False


def device_inputs(wl, device="cuda"):
    """x, ids and route weights of a synth MoE workload as device tensors."""
    x = torch.from_numpy(np.ascontiguousarray(wl.x).view(np.int16)).view(torch.float16)
    ids = torch.from_numpy(np.ascontiguousarray(wl.ids))
    wb = np.ascontiguousarray(wl.weights_bits)
    if wl.weights_dtype == "bf16":
        w = torch.from_numpy(wb.view(np.int16)).view(torch.bfloat16)
    elif wl.weights_dtype == "f16":
        w = torch.from_numpy(wb.view(np.int16)).view(torch.float16)
    else:
        w = torch.from_numpy(wb.astype(np.float32))
    return x.to(device), ids.to(device), w.to(device)


def f16_tensor(a, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float16).view(np.int16)).view(
        torch.float16).to(device)
