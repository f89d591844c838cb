"""CPU checks of the calls that carry rows to experts and back and of the
products with 4-bit weights: the oracles against closed forms and differences,
the tile layout, and every refusal of the C ABI and of the binding (nothing here
needs a GPU: pointers are numbers that fail the device check last)."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import permute as operm  # noqa: E402
from oracle import w4 as ow4  # noqa: E402
from trellis_quantized_moe_amd import exl3  # noqa: E402


# ------------------------------------------------------------------ oracles
def _pos(rng, T, k, dropped):
    pos = rng.permutation(T * k).reshape(T, k)
    pos[rng.random((T, k)) < dropped] = -1
    return pos


def test_gradient_oracle_against_differences():
    rng = np.random.default_rng(1)
    T, k, H = 5, 3, 4
    pos = _pos(rng, T, k, 0.3)
    y, w = rng.standard_normal((T * k, H)), rng.standard_normal((T, k))
    dout = rng.standard_normal((T, H))
    dy, dw = operm.unpermute_backward(dout, y, pos, w, np.zeros_like(y))
    step = 1e-6  # out is linear in y and in w: differences are exact but for rounding

    def loss(y, w):
        return float((dout * operm.unpermute(y, pos, w)).sum())

    for a, g in ((y, dy), (w, dw)):
        for i in np.ndindex(a.shape):
            hi, lo = a.copy(), a.copy()
            hi[i] += step
            lo[i] -= step
            d = (loss(hi, w) - loss(lo, w)) if a is y else (loss(y, hi) - loss(y, lo))
            assert abs(d / (2 * step) - g[i]) < 1e-8


def test_carrying_there_and_back():
    """Without weights a row comes back as often as it has choices, and the two
    calls are each other's transposes."""
    rng = np.random.default_rng(2)
    T, k, H = 7, 4, 3
    pos = _pos(rng, T, k, 0.2)
    x, y = rng.standard_normal((T, H)), rng.standard_normal((T * k, H))
    there = operm.permute(x, pos, np.zeros((T * k, H)))
    assert np.allclose(operm.unpermute(there, pos), x * (pos >= 0).sum(1)[:, None], rtol=1e-14)
    assert abs((there * y).sum() - (x * operm.unpermute(y, pos)).sum()) < 1e-12


def test_w4_oracle_against_dense():
    rng = np.random.default_rng(3)
    q = rng.integers(0, 256, (2, 3, 32), dtype=np.uint8)
    scale, zero = rng.random((2, 3, 2)), rng.integers(0, 16, (2, 3, 2))
    w = ow4.weights(q, scale, zero)
    x = rng.standard_normal((5, 64))
    out = ow4.linear(x, w, [0, 2, 4], np.full((5, 3), 9.0))
    for p, e in ((0, 0), (3, 1)):
        for n in range(3):
            want = sum(x[p, c] * scale[e, n, c // 32] *
                       (float(q[e, n, c // 2] >> (4 * (c % 2)) & 15) - zero[e, n, c // 32])
                       for c in range(64))
            assert abs(out[p, n] - want) < 1e-12
    assert np.all(out[4] == 9)


# ------------------------------------------------------------------- layout
@pytest.mark.parametrize("E,N,K,G,zeros", [(1, 8, 32, 32, True), (3, 24, 160, 32, True),
                                           (2, 40, 192, 64, False), (2, 16, 256, 128, True)])
def test_weight_tiles(E, N, K, G, zeros):
    g = torch.Generator().manual_seed(N)
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    scale = torch.randn(E, N, K // G, generator=g).to(torch.bfloat16)
    zero = torch.randint(0, 16, (E, N, K // G), generator=g, dtype=torch.uint8) if zeros else None
    W = exl3.DeviceW4(q, scale, zero)
    NT, KT, NG = (N + 15) // 16, (K + 127) // 128, 128 // G
    assert W.q.shape == (E, NT, KT, 64, 16) and W.scale.shape == (E, NT, KT, 16, NG)
    words = W.q.numpy().view(np.uint32)
    v = np.empty((E, N, K), np.uint8)
    v[:, :, 0::2], v[:, :, 1::2] = q.numpy() & 15, q.numpy() >> 4
    for e in range(E):
        for nt in range(NT):
            for kt in range(KT):
                for lane in range(64):
                    for i in range(4):
                        assert words[e, nt, kt, lane, i] == ow4.tile_word(v[e], nt, kt, lane, i)
                for gi in range(NG):
                    for n in range(16):
                        at = (e, 16 * nt + n, kt * NG + gi)
                        inside = at[1] < N and at[2] < K // G
                        assert float(W.scale[e, nt, kt, n, gi]) == (float(scale[at]) if inside
                                                                    else 0)
                        if zeros:
                            assert int(W.zero[e, nt, kt, n, gi]) == (int(zero[at]) if inside else 0)
    assert (W.zero is None) == (not zeros)
    c = W.cstruct()
    assert (c.in_features, c.out_features, c.num_experts, c.group_size) == (K, N, E, G)


def test_weights_that_lie_apart():
    """Slices at odd addresses, transposed and expanded tensors: the same tiles."""
    g = torch.Generator().manual_seed(1)
    q = torch.randint(0, 256, (3, 16, 32), generator=g, dtype=torch.uint8)
    s = torch.rand(3, 16, 2, generator=g).half().requires_grad_()
    want = exl3.DeviceW4(q, s)
    assert not want.scale.requires_grad
    odd = torch.empty(q.numel() + 3, dtype=torch.uint8)
    odd[3:] = q.reshape(-1)
    for other in (odd[3:].view(3, 16, 32), q.transpose(0, 2).contiguous().transpose(0, 2)):
        assert torch.equal(exl3.DeviceW4(other, s).q, want.q)
    one = exl3.DeviceW4(q[:1].expand(3, 16, 32), s[:1].expand(3, 16, 2))
    for e in range(3):
        assert torch.equal(one.q[e], want.q[0]) and torch.equal(one.scale[e], want.scale[0])


# ----------------------------------------------------------------- refusals
P = 1 << 20  # an address that is no device memory
FAR = 1 << 32


def _permute(x=P, dt=exl3.F16, ldx=256, rows=4, topk=2, features=256, pos=P, out=2 * P, ldo=256):
    return exl3.lib().exl3_permute(x, dt, ldx, rows, topk, features, pos, out, ldo, None, None)


BAD_MOVES = [
    (dict(rows=-1), -7), (dict(topk=0), -7), (dict(topk=33), -7), (dict(rows=(1 << 29) + 1), -7),
    (dict(features=0), -3), (dict(features=252), -3), (dict(features=65544, ldo=65544), -3),
    (dict(pos=None), -1), (dict(out=None), -1), (dict(ldo=248), -3), (dict(ldo=FAR + 8), -3),
    (dict(out=2 * P + 8), -4), (dict(ldo=260), -4), (dict(pos=P + 2), -4), (dict(), -5),
]


@pytest.mark.parametrize("kw,code", BAD_MOVES + [
    (dict(dt=exl3.I32), -2), (dict(dt=0), -2), (dict(x=None), -1), (dict(ldx=255), -3),
    (dict(ldx=FAR + 8), -3), (dict(x=P + 8), -4), (dict(ldx=258, dt=exl3.F32), -4),
    (dict(out=P), -7), (dict(dt=exl3.F32, ldx=260), -5),
    (dict(rows=0, x=None, pos=None, out=None), 0),
])
def test_permute_refusals(kw, code):
    assert _permute(**kw) == code


def _unpermute(y=P, y_dt=exl3.BF16, ldy=256, rows=4, topk=2, features=256, pos=P, w=P,
               w_dt=exl3.F32, out=2 * P, out_dt=exl3.F16, ldo=256):
    return exl3.lib().exl3_unpermute(y, y_dt, ldy, rows, topk, features, pos, w, w_dt, out, out_dt,
                                     ldo, None, None)


@pytest.mark.parametrize("kw,code", BAD_MOVES + [
    (dict(y_dt=exl3.I64), -2), (dict(out_dt=0), -2), (dict(w_dt=exl3.I32), -2), (dict(y=None), -1),
    (dict(ldy=248), -3), (dict(y=P + 4), -4), (dict(ldy=258), -4), (dict(w=P + 2), -4),
    (dict(out=P), -7), (dict(w=P + 2, w_dt=exl3.BF16), -5), (dict(w=None, w_dt=0), -5),
    (dict(out_dt=exl3.F32, ldo=260), -5), (dict(rows=0, y=None, pos=None, w=None, out=None), 0),
])
def test_unpermute_refusals(kw, code):
    assert _unpermute(**kw) == code


def _backward(dout=P, do_dt=exl3.F32, ldd=256, rows=4, topk=2, features=256, pos=P, y=2 * P,
              y_dt=exl3.F16, ldy=256, w=P, w_dt=exl3.F32, out=4 * P, ldo=256, dw=8 * P,
              dw_dt=exl3.F32):
    return exl3.lib().exl3_unpermute_backward(dout, do_dt, ldd, rows, topk, features, pos, y, y_dt,
                                              ldy, w, w_dt, out, ldo, dw, dw_dt, None, None)


@pytest.mark.parametrize("kw,code", BAD_MOVES + [
    (dict(do_dt=exl3.I32), -2), (dict(y_dt=0), -2), (dict(w_dt=0), -2), (dict(dw_dt=0), -2),
    (dict(dout=None), -1), (dict(y=None), -1), (dict(dw=None), -1), (dict(ldd=248), -3),
    (dict(ldy=248), -3), (dict(dout=P + 8), -4), (dict(ldd=258), -4), (dict(y=P + 8), -4),
    (dict(w=P + 2), -4), (dict(dw=8 * P + 2), -4), (dict(out=P), -7), (dict(out=2 * P), -7),
    (dict(dw=P), -7), (dict(y=None, dw=None, ldy=0, dw_dt=0), -5), (dict(w=None, w_dt=0), -5),
    (dict(dw=8 * P + 2, dw_dt=exl3.F16), -5),
    (dict(rows=0, dout=None, y=None, pos=None, w=None, out=None, dw=None), 0),
])
def test_unpermute_backward_refusals(kw, code):
    assert _backward(**kw) == code


def _w4(weight="default", x=P, dt=exl3.F16, ldx=256, rows=4, offset=P, out=2 * P, out_dt=exl3.F32,
        ldo=128, **kw):
    d = dict(in_features=256, out_features=128, num_experts=3, group_size=64, q=P, scale=P, zero=P,
             scale_dtype=exl3.F16)
    d.update(kw)
    c = exl3.W4C(*[d[n] for n, _ in exl3.W4C._fields_]) if weight == "default" else weight
    return exl3.lib().exl3_w4_linear(ctypes.byref(c) if c else None, x, dt, ldx, rows, offset, out,
                                     out_dt, ldo, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(weight=None), -1), (dict(q=None), -1), (dict(scale=None), -1), (dict(x=None), -1),
    (dict(out=None), -1), (dict(offset=None), -1), (dict(rows=-1), -7),
    (dict(rows=(1 << 30) + 1), -7), (dict(num_experts=0), -7), (dict(num_experts=1025), -7),
    (dict(group_size=0), -7), (dict(group_size=16), -7), (dict(group_size=256), -7),
    (dict(in_features=0), -3), (dict(in_features=288), -3), (dict(in_features=65600), -3),
    (dict(out_features=0), -3), (dict(out_features=132), -3), (dict(out_features=65544), -3),
    (dict(dt=exl3.F32), -2), (dict(scale_dtype=exl3.F32), -2), (dict(out_dt=exl3.I32), -2),
    (dict(ldx=248), -3), (dict(ldo=120), -3), (dict(ldx=FAR + 8), -3), (dict(ldo=FAR + 8), -3),
    (dict(x=P + 8), -4), (dict(out=2 * P + 8), -4), (dict(q=P + 8), -4), (dict(scale=P + 8), -4),
    (dict(zero=P + 8), -4), (dict(offset=P + 2), -4), (dict(ldx=260), -4), (dict(ldo=130), -4),
    (dict(out=P), -7), (dict(), -5), (dict(zero=None), -5), (dict(num_experts=1, offset=None), -5),
    (dict(dt=exl3.BF16, scale_dtype=exl3.BF16, out_dt=exl3.F16, ldo=136), -5),
    (dict(rows=0, x=None, q=None, out=None, offset=None), 0),
])
def test_w4_refusals(kw, code):
    assert _w4(**kw) == code


def test_binding_refuses_wrong_shapes_and_layouts():
    E = exl3.Exl3Error
    meta = {"pos_of_pair": torch.zeros(8, dtype=torch.int32)}
    x, y = torch.zeros(4, 16), torch.zeros(8, 16)
    for bad in (dict(x=x.t()), dict(x=x[0]), dict(topk=0), dict(topk=3), dict(topk=1 << 40),
                dict(out=y[:7]), dict(out=y.half()), dict(out=torch.zeros(16, 8).t()),
                dict(meta={"pos_of_pair": torch.zeros(8, dtype=torch.int64)}),
                dict(meta={"pos_of_pair": torch.zeros(16, dtype=torch.int32)[::2]})):
        with pytest.raises(E):
            exl3.exl3_permute(**{**dict(x=x, meta=meta, topk=2), **bad})
    w = torch.zeros(4, 2)
    for bad in (dict(y=y[:7]), dict(y=y[0]), dict(topk=0), dict(w=w.t()), dict(w=w[:3]),
                dict(out=y), dict(out=x.t())):
        with pytest.raises(E):
            exl3.exl3_unpermute(**{**dict(y=y, meta=meta, topk=2, w=w), **bad})
    for bad in (dict(dout=x[0]), dict(y=y[:7]), dict(y=y.half(), dy=y), dict(w=w.t()),
                dict(dw=w[:3]), dict(dy=y[:7]), dict(y=None, dw=w)):
        with pytest.raises(E):
            exl3.exl3_unpermute_backward(**{**dict(dout=x, meta=meta, topk=2, y=y, w=w), **bad})
    q = torch.zeros(2, 8, 32, dtype=torch.uint8)
    s, z = torch.zeros(2, 8, 2, dtype=torch.float16), torch.zeros(2, 8, 2, dtype=torch.uint8)
    for bad in (dict(q=q.int()), dict(q=q[0, 0]), dict(q=q[:, :0]), dict(scale=s.float()),
                dict(scale=s[:, :, :0]), dict(scale=s[:, :7]),
                dict(scale=torch.zeros(2, 8, 3, dtype=torch.float16)), dict(zero=z[:1]),
                dict(zero=z.int()), dict(zero=z + 16)):
        with pytest.raises(E):
            exl3.DeviceW4(**{**dict(q=q, scale=s, zero=z), **bad})
    W = exl3.DeviceW4(q, s, z)
    off, xh = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 64, dtype=torch.float16)
    for bad in (dict(x=xh[0]), dict(x=xh[:, :32]), dict(x=torch.zeros(64, 4).half().t()),
                dict(expert_offset=off[:2]), dict(expert_offset=off.long()),
                dict(out=torch.zeros(4, 9)), dict(out=torch.zeros(3, 8))):
        with pytest.raises(E):
            exl3.exl3_w4_linear(**{**dict(x=xh, weight=W, expert_offset=off), **bad})


def test_binding_refuses_sizes_past_32_bits():
    """Cut off to 32 bits, only the first rows would be worked on."""
    far = torch.empty(1, 8, dtype=torch.float16).expand(FAR + 4, 8)
    meta = {"pos_of_pair": torch.empty(1, dtype=torch.int32).expand(FAR + 4)}
    W = exl3.DeviceW4(torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(8, 1).half())
    for call in (lambda: exl3.exl3_permute(far, meta, 1), lambda: exl3.exl3_unpermute(far, meta, 1),
                 lambda: exl3.exl3_unpermute_backward(far, meta, 1),
                 lambda: exl3.exl3_w4_linear(far, W)):
        with pytest.raises(exl3.Exl3Error, match="out of range"):
            call()
