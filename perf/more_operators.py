"""Workloads of the operators that carry rows to experts and back, and of the
experts' products with 4-bit weights.

``run`` computes a case from elementary torch operations, or, where ``own`` is
true, through ``trellis_quantized_moe_amd.exl3``. ``exact`` is the same result
in 64 bits, from the definitions.

Definitions. Row t has k choices (t, j); pos(t, j) is the place of that pair
among all pairs in ascending order of (expert, pair), -1 where the choice names
no expert. Places past the last pair keep what they held.
  permute    xs[pos(t, j)] = x[t]
  unpermute  out[t] = sum_j w[t, j] y[pos(t, j)]; without w all weights are 1,
             which is the gradient of permute
  backward   of unpermute: dy[pos(t, j)] = w[t, j] dout[t] and
             dw[t, j] = sum_h dout[t, h] y[pos(t, j), h] (0 where pos is -1)
  w4         out[p, n] = sum_k x[p, k] s[e, n, k // g] (q[e, n, k] - z[e, n, k // g])
             for the sorted rows p of expert e; q has 4 bits, z as well (8 where
             there are no zeros), g is the group size. One expert: all rows.
"""

import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _move(name, op, tokens, experts, topk, features, x, w, out, pad, masked):
    """x: type of the rows that come in; w: of the weights; out: of what goes out."""
    return dict(name=name, op=op, tokens=tokens, experts=experts, topk=topk, features=features,
                x=x, w=w, out=out, pad=pad, masked=masked)


def _w4(name, tokens, experts, topk, fin, fout, group, zeros, x, scale, out, pad):
    """experts 0: one projection for all rows (topk 1)."""
    return dict(name=name, op="w4", tokens=tokens, experts=experts, topk=topk, fin=fin, fout=fout,
                group=group, zeros=zeros, x=x, scale=scale, out=out, pad=pad)


def listed():
    return [
        # a decode batch on its way to 128 experts
        _move("permute_batch", "permute", 61, 128, 8, 4096, "f16", "none", "f16", 0, False),
        # prompt rows of the 192-expert layer, the last tenth of them padding
        _move("permute_prompt", "permute", 8192, 192, 8, 6144, "bf16", "none", "bf16", 0, True),
        # one token's results of the 128-expert decode layer
        _move("unpermute_token", "unpermute", 1, 128, 8, 4096, "f16", "f32", "f16", 0, False),
        # prompt results in 32 bits, written into a column slice of a wider buffer
        _move("unpermute_prompt", "unpermute", 4001, 192, 8, 6144, "f32", "f16", "bf16", 64, True),
        # gradient of a training step's sorting: no weights
        _move("permute_gradient", "unpermute", 2047, 128, 8, 4096, "bf16", "none", "f32", 0, False),
        # gradients of a small training step's results and route weights
        _move("backward_step", "backward", 2047, 128, 8, 4096, "bf16", "f32", "bf16", 0, True),
        # gradients of a long batch
        _move("backward_long", "backward", 8192, 256, 4, 6144, "f16", "f16", "f32", 0, False),
        # one token through one projection
        _w4("w4_token", 1, 0, 1, 4096, 4096, 128, False, "f16", "f16", "f16", 0),
        # one token through its eight experts
        _w4("w4_experts_token", 1, 128, 8, 4096, 1536, 128, False, "bf16", "bf16", "f32", 0),
        # a decode batch over 192 experts, small groups with their own zeros
        _w4("w4_experts_batch", 61, 192, 8, 6144, 2048, 32, True, "f16", "f16", "f16", 0),
        # a prompt through one projection, x a column slice of a wider buffer
        _w4("w4_prompt", 4001, 0, 1, 6144, 4096, 64, True, "bf16", "f16", "bf16", 64),
        # a prompt's pairs through the second product of 128 experts
        _w4("w4_experts_prompt", 4096, 128, 8, 1536, 4096, 128, False, "f16", "f16", "f32", 0),
    ]


MOST_MOVED = 8192 * 8 * 6144  # values of the largest listed move
MOST_MACS = 4096 * 8 * 1536 * 4096
MOST_WEIGHTS = 192 * 6144 * 2048


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "unpermute", "backward", "w4", "w4", "w4"])
    experts = rng.choice([8, 16, 60, 128, 192, 256, rng.randint(2, 512)])
    types = ["f16", "bf16"]
    if op != "w4":
        topk = rng.randint(1, min(experts, 16))
        features = rng.choice([512, 1536, 2048, 4096, 6144, 8 * rng.randint(8, 1024)])
        tokens = min(_log(rng, 1, 16384), MOST_MOVED // (2 * topk * features))
        x = rng.choice(types + ["f32"])
        c = _move("", op, tokens, experts, topk, features, x,
                  "none" if op == "permute" else rng.choice(types + ["f32"]),
                  x if op == "permute" else rng.choice(types + ["f32"]),
                  rng.choice([0, 0, 64]), rng.random() < 0.4)
        if op == "unpermute" and rng.random() < 0.3:
            c["w"] = "none"
    else:
        group = rng.choice([32, 64, 128])
        fin = group * max(1, _log(rng, 256, 8192) // group)
        fout = rng.choice([192, 512, 1536, 2048, 4096, 6144, 8 * rng.randint(8, 1024)])
        if rng.random() < 0.5:
            experts, topk = 0, 1
        else:
            experts = max(1, min(experts, MOST_WEIGHTS // (fin * fout)))
            topk = rng.randint(1, min(experts, 8))
        tokens = max(1, min(_log(rng, 1, 16384), MOST_MACS // (topk * fin * fout)))
        c = _w4("", tokens, experts, topk, fin, fout, group, rng.random() < 0.5, rng.choice(types),
                rng.choice(types), rng.choice(types + ["f32"]), rng.choice([0, 0, 64]))
    del c["name"]
    return c


def _live(case):
    """Rows that are not padding."""
    T = case["tokens"]
    return max(1, T - max(1, T // 10)) if case["masked"] else T


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2, "none": 0}
    P = case["tokens"] * case["topk"]
    if case["op"] == "w4":
        K, N, g = case["fin"], case["fout"], case["group"]
        E, share = case["experts"], case["topk"] / max(1, case["experts"])
        # experts that a batch of this size meets, their routes spread evenly
        used = E * (1 - (1 - share) ** case["tokens"]) if E else 1
        per_weight = 0.5 + (3 if case["zeros"] else 2) / g
        return {"bytes": used * N * K * per_weight + P * K * 2 + P * N * size[case["out"]],
                "flops": 2 * P * N * K}
    T, H = case["tokens"], case["features"]
    kept = _live(case) * case["topk"]
    x, w, out = size[case["x"]], size[case["w"]], size[case["out"]]
    if case["op"] == "permute":
        return {"bytes": _live(case) * H * x + kept * H * x + 4 * P, "flops": kept * H}
    if case["op"] == "unpermute":
        return {"bytes": kept * H * x + T * H * out + P * (4 + w), "flops": 2 * kept * H}
    return {"bytes": _live(case) * H * out + 2 * kept * H * x + P * (4 + 2 * w),
            "flops": 3 * kept * H}


# ------------------------------------------------------------------ inputs
def _normal(g, rows, cols, pad, dtype):
    """Normal values [rows][cols], a column slice of a buffer `pad` wider."""
    return torch.randn(rows, cols + pad, generator=g, device="cuda").to(dtype)[:, :cols]


def _routes(g, case, live):
    """Routes of the tokens and where their pairs stand when sorted by expert."""
    T, E, k = case["tokens"], case["experts"], case["topk"]
    ids = torch.topk(torch.randn(T, E, generator=g, device="cuda"), k, dim=1).indices
    ids[live:] = E
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device="cuda")
    gone = flat == E
    count = torch.bincount(flat, minlength=E + 1)[:E]
    offset = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offset[1:] = count.cumsum(0)
    return {"expert_count": count.to(torch.int32), "expert_offset": offset.to(torch.int32),
            "pair_of_pos": torch.where(gone[order], -1, order).to(torch.int32),
            "pos_of_pair": torch.where(gone, -1, pos).to(torch.int32)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    T, k = case["tokens"], case["topk"]
    if case["op"] == "w4":
        E, K, N, n = max(1, case["experts"]), case["fin"], case["fout"], case["group"]
        s["offset"] = None
        if case["experts"]:
            s["offset"] = _routes(g, case, T)["expert_offset"]
        s["x"] = _normal(g, T * k, K, case["pad"], DT[case["x"]])
        # two weights a byte, the lower four bits first
        s["q"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda",
                               dtype=torch.uint8)
        spread = torch.rand(E, N, K // n, generator=g, device="cuda")
        s["scale"] = ((0.5 + spread) / (4.6 * math.sqrt(K))).to(DT[case["scale"]])
        s["zero"] = None
        if case["zeros"]:
            s["zero"] = torch.randint(0, 16, (E, N, K // n), generator=g, device="cuda",
                                      dtype=torch.uint8)
        if own:
            from trellis_quantized_moe_amd import exl3
            s["weight"] = exl3.DeviceW4(s["q"], s["scale"], s["zero"])
        return s
    H, P, live = case["features"], T * k, _live(case)
    s["meta"] = _routes(g, case, live)
    kind, x, out = case["op"], DT[case["x"]], DT[case["out"]]
    s["w"] = None
    if case["w"] != "none":
        w = torch.rand(T, k, generator=g, device="cuda") + 0.1
        s["w"] = (w / w.sum(1, keepdim=True)).to(DT[case["w"]])
    # the buffers that the results go to: places past the last pair stay 0
    if kind == "permute":
        s["x"] = _normal(g, T, H, case["pad"], x)
        s["out"] = torch.zeros(P, H, dtype=x, device="cuda")
    else:
        s["y"] = _normal(g, P, H, 0, x)
        if kind == "unpermute":
            s["out"] = torch.zeros(T, H + case["pad"], dtype=out, device="cuda")[:, :H]
        else:
            s["dout"] = _normal(g, T, H, case["pad"], out)
            s["dy"] = torch.zeros(P, H, dtype=x, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _rows_of_places(s):
    """Row of each place, and which places hold a pair."""
    pair = s["meta"]["pair_of_pos"].long()
    return torch.where(pair >= 0, pair, 0) // s["case"]["topk"], (pair >= 0)[:, None]


def _plain_permute(s):
    row, held = _rows_of_places(s)
    return torch.where(held, s["x"][row], 0)


def _plain_unpermute(s):
    case = s["case"]
    pos = s["meta"]["pos_of_pair"].long().reshape(case["tokens"], case["topk"])
    total = torch.zeros(case["tokens"], case["features"], device=pos.device)
    for j in range(case["topk"]):
        y = s["y"][pos[:, j].clamp(min=0)].float()
        if s["w"] is not None:
            y = y * s["w"][:, j:j + 1].float()
        total += torch.where(pos[:, j:j + 1] >= 0, y, 0.0)
    return total.to(DT[case["out"]])


def _plain_backward(s):
    case = s["case"]
    row, held = _rows_of_places(s)
    weight = s["w"].float().reshape(-1)[s["meta"]["pair_of_pos"].long().clamp(min=0)]
    dy = torch.where(held, weight[:, None] * s["dout"].float()[row], 0.0)
    pos = s["meta"]["pos_of_pair"].long().reshape(case["tokens"], case["topk"])
    dw = torch.stack([(s["dout"].float() * s["y"][pos[:, j].clamp(min=0)].float()).sum(1)
                      for j in range(case["topk"])], dim=1)
    return {"dy": dy.to(s["dy"].dtype), "dw": torch.where(pos >= 0, dw, 0.0).to(s["w"].dtype)}


def _plain_w4(s):
    case = s["case"]
    K, N, n = case["fin"], case["fout"], case["group"]
    ends = [0, case["tokens"]]
    if s["offset"] is not None:
        ends = s["offset"].tolist()
    out = torch.empty(case["tokens"] * case["topk"], N, dtype=DT[case["out"]],
                      device=s["x"].device)
    for e in range(len(ends) - 1):
        if ends[e] == ends[e + 1]:
            continue
        q = torch.stack([s["q"][e] & 15, s["q"][e] >> 4], dim=-1).reshape(N, K // n, n).float()
        zero = 8.0 if s["zero"] is None else s["zero"][e].float()[:, :, None]
        w = ((q - zero) * s["scale"][e].float()[:, :, None]).reshape(N, K)
        out[ends[e]:ends[e + 1]] = (s["x"][ends[e]:ends[e + 1]].float() @ w.t()).to(out.dtype)
    return out


# --------------------------------------------------------------------- run
def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"permute": _plain_permute, "unpermute": _plain_unpermute,
                "backward": _plain_backward, "w4": _plain_w4}[op](state)
    from trellis_quantized_moe_amd import exl3
    if op == "w4":
        return exl3.exl3_w4_linear(state["x"], state["weight"], expert_offset=state["offset"],
                                   out_dtype=DT[case["out"]])
    if op == "permute":
        return exl3.exl3_permute(state["x"], state["meta"], case["topk"], out=state["out"])
    if op == "unpermute":
        return exl3.exl3_unpermute(state["y"], state["meta"], case["topk"], w=state["w"],
                                   out=state["out"])
    dy, dw = exl3.exl3_unpermute_backward(state["dout"], state["meta"], case["topk"],
                                          y=state["y"], w=state["w"], dy=state["dy"])
    return {"dy": dy, "dw": dw}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    T, k = case["tokens"], case["topk"]
    if case["op"] == "w4":
        E, N, K, n = max(1, case["experts"]), case["fout"], case["fin"], case["group"]
        result = torch.zeros(T * k, N, dtype=torch.float64, device="cuda")
        bounds = [0, T] if s["offset"] is None else s["offset"].cpu().tolist()
        for e in range(E):
            a, b = bounds[e], bounds[e + 1]
            if a == b:
                continue
            w = torch.empty(N, K, dtype=torch.float64, device="cuda")
            w[:, 0::2] = (s["q"][e] % 16).double()
            w[:, 1::2] = torch.div(s["q"][e], 16, rounding_mode="floor").double()
            w -= 8 if s["zero"] is None else s["zero"][e].double().repeat_interleave(n, 1)
            w *= s["scale"][e].double().repeat_interleave(n, 1)
            result[a:b] = torch.mm(s["x"][a:b].double(), w.t().contiguous())
        return result
    pos = s["meta"]["pos_of_pair"].long()
    pair = torch.nonzero(pos >= 0).flatten()
    place, token = pos[pair], pair // k
    H = case["features"]
    weight = torch.ones(T * k, dtype=torch.float64, device="cuda")
    if s["w"] is not None:
        weight = s["w"].double().flatten()
    if case["op"] == "unpermute":
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for i in range(0, H, 512):  # a few columns at a time
            part = weight[pair, None] * s["y"][place, i:i + 512].double()
            out[:, i:i + 512] = out[:, i:i + 512].index_add(0, token, part)
        return out
    if case["op"] == "permute":
        out = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        out[place] = s["x"][token].double()
        return out
    dy = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    for i in range(0, H, 512):
        d = s["dout"][:, i:i + 512].double()[token]
        dy[place, i:i + 512] = weight[pair, None] * d
        dw[pair] += (d * s["y"][place, i:i + 512].double()).sum(1)
    return {"dy": dy, "dw": dw.reshape(T, k)}
