"""What is measured of the mixture-of-experts operators: routing, the products of rows with the NVFP4
weights of the experts picked for them, and the experts' SwiGLU layer, each with its plain form.

Three operators (a case's "op"):

* "route":  scores of E experts per row -> the ids of the top_k experts and their weights;
* "linear": y[i, j] = W[ids[i, j]] x[i] over NVFP4 weights (E2M1 codes, an E4M3 scale per 16 along K, a tensor scale per expert);
* "moe":    out[i] = sum_j w[i, j] * down_e(silu(gate_e(x[i])) * up_e(x[i])), e = ids[i, j].

Weights are drawn in NVFP4 directly: codes of normal values, scales around one.  The ids of "linear" and "moe" come from
a router whose experts differ in popularity; a share of the rows may be padding (ids -1).
"""
import math

import torch

own = False

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step: the latency of the router
        {"name": "route one row", "op": "route", "m": 1, "experts": 64, "top_k": 8, "scoring": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_score": "max", "renormalize": True, "scale": 1.0, "logits": "float32", "masked": 0.0},
        # a decode batch of a model with grouped experts, sigmoid scores and a balancing bias
        {"name": "route grouped sigmoid", "op": "route", "m": 509, "experts": 256, "top_k": 8, "scoring": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_score": "top2", "renormalize": True, "scale": 2.5, "logits": "float32", "masked": 0.0},
        # a long prompt, bf16 logits (many equal ones), some experts masked out
        {"name": "route prompt bf16", "op": "route", "m": 16384, "experts": 128, "top_k": 8, "scoring": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_score": "max", "renormalize": False, "scale": 1.0, "logits": "bfloat16", "masked": 0.05},
        # matrix-vector products of one token with its experts' weights
        {"name": "linear one row", "op": "linear", "m": 1, "experts": 64, "top_k": 8, "n": 2048, "k": 1024, "padding": 0.0},
        # a ragged decode batch, sizes that are no multiple of a tile
        {"name": "linear ragged", "op": "linear", "m": 37, "experts": 20, "top_k": 3, "n": 1000, "k": 1056, "padding": 0.1},
        # a prompt through one projection
        {"name": "linear prompt", "op": "linear", "m": 2048, "experts": 32, "top_k": 4, "n": 2048, "k": 2048, "padding": 0.0},
        # decode of one token: many small experts
        {"name": "moe one row, small experts", "op": "moe", "m": 1, "experts": 64, "top_k": 8, "hidden": 2048, "inter": 1024, "padding": 0.0},
        # decode of one token: few large experts (hidden and inter of the fixed-format workload)
        {"name": "moe one row, large experts", "op": "moe", "m": 1, "experts": 8, "top_k": 2, "hidden": 4096, "inter": 12288, "padding": 0.0},
        # a decode batch: nearly every expert is used, a few rows each
        {"name": "moe 32 rows", "op": "moe", "m": 32, "experts": 64, "top_k": 8, "hidden": 2048, "inter": 1024, "padding": 0.0},
        # a padded batch of odd sizes
        {"name": "moe ragged", "op": "moe", "m": 203, "experts": 20, "top_k": 3, "hidden": 1056, "inter": 672, "padding": 0.2},
        # a short prompt over few large experts
        {"name": "moe 512 rows, large experts", "op": "moe", "m": 512, "experts": 8, "top_k": 2, "hidden": 4096, "inter": 12288, "padding": 0.0},
        # a long prompt over many small experts
        {"name": "moe prompt", "op": "moe", "m": 4096, "experts": 64, "top_k": 8, "hidden": 2048, "inter": 1024, "padding": 0.0},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over their logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["route", "linear", "linear", "moe", "moe", "moe"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 8, 512 // groups)
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, top_groups * (experts // groups)))
        return {"op": op, "m": _log(rng, 1, 16384), "experts": experts, "top_k": top_k, "scoring": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups, "group_score": rng.choice(["max", "top2"]),
                "renormalize": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "logits": rng.choice(["float32", "bfloat16"]),
                "masked": rng.choice([0.0, 0.0, 0.1])}
    while True:
        experts = _log(rng, 4, 128)
        top_k = rng.randint(1, min(8, experts))
        case = {"op": op, "m": _log(rng, 1, 4096), "experts": experts, "top_k": top_k, "padding": rng.choice([0.0, 0.0, 0.15])}
        if op == "linear":
            case.update(n=_log(rng, 64, 4096), k=32 * _log(rng, 4, 128))
            weights = experts * case["n"] * case["k"]
        else:
            case.update(hidden=32 * _log(rng, 8, 128), inter=32 * _log(rng, 4, 192))
            weights = 3 * experts * case["hidden"] * case["inter"]
        if weights <= 4 * 10**8 and 2 * case["m"] * top_k * weights / experts <= 4 * 10**11:
            return case


# ------------------------------------------------------------------ inputs

def _experts_weight(g, experts, n, k, parts):
    """Codes uint8 [E, n, k/2] (element 2j in the low nibble), E4M3 scale bytes [E, n, k/16], tensor scales [E, parts]."""
    magnitude = torch.empty((experts, n, k // 2), device="cuda")

    def code():
        v = magnitude.normal_(0.0, 2.2, generator=g)
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        return torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)

    codes = code()
    codes |= code() << 4
    scales = torch.empty((experts, n, k // 16), device="cuda").log_normal_(3.0, 0.4, generator=g).clamp_(2.0**-6, 448.0)
    scales = scales.to(torch.float8_e4m3fn).view(torch.uint8)
    gs = torch.empty((experts, parts), device="cuda").uniform_(0.5, 2.0, generator=g) * (1.0 / (60.0 * math.sqrt(k)))
    return codes, scales, gs


def _ids(g, case):
    """Each row's top_k experts, some experts more popular than others; padding rows hold -1."""
    m, experts, top_k = case["m"], case["experts"], case["top_k"]
    logits = torch.randn((m, experts), generator=g, device="cuda") + 0.7 * torch.randn((experts,), generator=g, device="cuda")
    s, ids = torch.topk(torch.softmax(logits, dim=1), top_k, dim=1)
    ids = ids.to(torch.int32)
    ids[torch.rand((m,), generator=g, device="cuda") < case["padding"]] = -1
    return ids, s / s.sum(dim=1, keepdim=True)


def _inputs(case, seed):
    """Everything that a program has before it builds handles and buffers."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    m = case["m"]
    if case["op"] == "route":
        e = case["experts"]
        logits = 1.5 * torch.randn((m, e), generator=g, device="cuda") + 0.5 * torch.randn((e,), generator=g, device="cuda")
        logits[torch.rand((m, e), generator=g, device="cuda") < case["masked"]] = -math.inf
        s["logits"] = logits.to(getattr(torch, case["logits"])).contiguous()
        s["bias"] = 0.05 * torch.randn((e,), generator=g, device="cuda") if case["bias"] else None
        return s
    s["ids"], s["weights"] = _ids(g, case)
    s["x"] = torch.randn((m, case["k"] if case["op"] == "linear" else case["hidden"]), generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] == "linear":
        s["w"] = _experts_weight(g, case["experts"], case["n"], case["k"], 1)
    else:
        s["gate_up"] = _experts_weight(g, case["experts"], 2 * case["inter"], case["hidden"], 2)
        s["down"] = _experts_weight(g, case["experts"], case["hidden"], case["inter"], 1)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from nvfp4_quantized_dense_w4a16_b200 import native as N
        m, k = case["m"], case["top_k"]
        if case["op"] == "route":
            s["ids"] = torch.empty((m, k), dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty((m, k), dtype=torch.float32, device="cuda")
            return s
        if case["op"] == "linear":
            codes, scales, gs = s["w"]
            s["w"] = N.ffn_nvfp4_experts_create(codes, scales, gs)
            s["out"] = torch.empty((m, k, case["n"]), dtype=torch.bfloat16, device="cuda")
            size = N.ffn_nvfp4_experts_workspace_size(m, k, case["experts"], case["n"], case["k"])
        else:
            s["gate_up"] = N.ffn_nvfp4_experts_create(*s["gate_up"], gate_up=True)
            s["down"] = N.ffn_nvfp4_experts_create(*s["down"])
            s["out"] = torch.empty((m, case["hidden"]), dtype=torch.bfloat16, device="cuda")
            size = N.ffn_nvfp4_moe_workspace_size(m, k, case["experts"], case["hidden"], case["inter"])
        s["workspace"] = torch.empty((max(16, size),), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _plain_route(s):
    # 64 bits: two keys that differ by less than an fp32 step decide which expert is chosen
    c = s["case"]
    m, e, k = c["m"], c["experts"], c["top_k"]
    logits = s["logits"].double()
    log_s = logits - torch.logsumexp(logits, dim=1, keepdim=True) if c["scoring"] == "softmax" else -torch.log1p(torch.exp(-logits))
    key = torch.exp(log_s)
    if s["bias"] is not None:
        key = key + s["bias"].double()
    key = torch.where(torch.isinf(logits), -math.inf, key)
    if c["groups"] > 1:
        grouped = key.reshape(m, c["groups"], e // c["groups"])
        best = torch.sort(grouped, dim=2, descending=True).values
        group = best[:, :, 0]
        if c["group_score"] == "top2" and e // c["groups"] > 1:
            group = group + torch.where(torch.isinf(best[:, :, 1]), 0.0, best[:, :, 1])
        chosen = torch.sort(group, dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, chosen, True)
        key = torch.where(keep[:, :, None], grouped, -math.inf).reshape(m, e)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    there = top > -math.inf
    log_w = torch.where(there, log_s.gather(1, ids), -math.inf)
    if c["renormalize"]:
        log_w = log_w - torch.logsumexp(log_w, dim=1, keepdim=True)
    w = torch.where(there, c["scale"] * torch.exp(log_w), 0.0)
    return {"ids": torch.where(there, ids, -1).to(torch.int32), "weights": w.float()}


def _plain_dequant(codes, scales, gs):
    """fp32 weights [E, n, k] of the experts given; gs [E, 1] or, for gate and up, [E, 2]."""
    magnitude = torch.tensor(_MAGNITUDES, device=codes.device)
    value = torch.cat([magnitude, -magnitude])
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([value[byte & 15], value[byte >> 4]], dim=1)
    e, n, half = codes.shape
    w = pairs[codes.int()].reshape(e, n, half // 8, 16)
    w = w * scales.view(torch.float8_e4m3fn).float()[:, :, :, None]
    parts = gs.shape[1]
    return w.reshape(e, parts, n // parts, 2 * half).mul_(gs[:, :, None, None]).reshape(e, n, 2 * half)


def _plain_group(ids):
    """The (row, slot) pairs grouped by expert: the experts used, and each pair's group and place in it (padding: a group of its own)."""
    flat = ids.reshape(-1).long()
    used, group, counts = torch.unique(flat, return_inverse=True, return_counts=True)
    order = torch.argsort(group, stable=True)
    start = torch.cumsum(counts, 0) - counts
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device=flat.device) - start[group[order]]
    return used, group, place, int(counts.max())


def _plain_linear(x, top_k, ids, w):
    """fp32 [m, top_k, n]: every pair's row times its expert's weight."""
    m = x.shape[0]
    used, group, place, most = _plain_group(ids)
    rows = x.float().repeat_interleave(top_k, dim=0)
    padded = rows.new_zeros((used.numel(), most, rows.shape[1]))
    padded[group, place] = rows
    pick = used.clamp(min=0)
    y = torch.bmm(padded, _plain_dequant(w[0][pick], w[1][pick], w[2][pick]).transpose(1, 2))[group, place]
    y = torch.where((ids.reshape(-1) >= 0)[:, None], y, 0.0)
    return y.reshape(m, -1, y.shape[1])


def run(s):
    c = s["case"]
    if own:
        from nvfp4_quantized_dense_w4a16_b200 import native as N
        if c["op"] == "route":
            ids, weights = N.ffn_nvfp4_moe_route(s["logits"], c["top_k"], scoring=c["scoring"], bias=s["bias"], groups=c["groups"],
                                                 top_groups=c["top_groups"], group_score=c["group_score"],
                                                 renormalize=c["renormalize"], scale=c["scale"], ids=s["ids"], weights=s["weights"])
            return {"ids": ids, "weights": weights}
        if c["op"] == "linear":
            return N.ffn_nvfp4_experts_linear(s["x"], s["w"], s["ids"], y=s["out"], workspace=s["workspace"])
        return N.ffn_nvfp4_moe_forward(s["x"], s["gate_up"], s["down"], s["ids"], s["weights"], out=s["out"], workspace=s["workspace"])
    if c["op"] == "route":
        return _plain_route(s)
    if c["op"] == "linear":
        return _plain_linear(s["x"], c["top_k"], s["ids"], s["w"]).to(torch.bfloat16)
    gate_up = _plain_linear(s["x"], c["top_k"], s["ids"], s["gate_up"])
    gate, up = gate_up.chunk(2, dim=2)
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = _plain_linear(h.reshape(-1, h.shape[2]), 1, s["ids"].reshape(-1, 1), s["down"]).reshape(c["m"], c["top_k"], -1)
    return (s["weights"][:, :, None] * y).sum(dim=1).to(torch.bfloat16)


# ------------------------------------------------------------------ floors and exact values

def _used(case):
    """Experts that m rows of top_k picks are expected to touch."""
    rows = case["m"] * (1.0 - case["padding"])
    return case["experts"] * (1.0 - (1.0 - case["top_k"] / case["experts"]) ** rows)


def work(case):
    m, k = case["m"], case["top_k"]
    if case["op"] == "route":
        e = case["experts"]
        return {"bytes": m * e * (4 if case["logits"] == "float32" else 2) + 4 * e * case["bias"] + 8 * m * k, "flops": 8 * m * e}
    rows = m * k * (1.0 - case["padding"])
    if case["op"] == "linear":
        weight = case["n"] * case["k"]
        return {"bytes": 0.5625 * weight * _used(case) + 2 * m * case["k"] + 4 * m * k + 2 * m * k * case["n"], "flops": 2 * rows * weight}
    weight = 3 * case["hidden"] * case["inter"]
    return {"bytes": 0.5625 * weight * _used(case) + 4 * m * case["hidden"] + 8 * m * k, "flops": 2 * rows * weight}


def _exact_weight(w, e):
    """One expert's weights in 64 bits, [parts, n / parts, k], from the bits of the format."""
    codes, scales, gs = (t[e] for t in w)
    nibble = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(codes.shape[0], -1).to(torch.int32)
    exponent, mantissa = (nibble >> 1) & 3, (nibble & 1).double()
    value = torch.where(exponent == 0, 0.5 * mantissa, (1.0 + 0.5 * mantissa) * torch.exp2(exponent.double() - 1.0))
    value = torch.where(nibble >= 8, -value, value)
    b = scales.to(torch.int32)
    exponent, mantissa = (b >> 3) & 15, (b & 7).double()
    scale = torch.where(exponent == 0, mantissa / 512.0, (1.0 + mantissa / 8.0) * torch.exp2(exponent.double() - 7.0))
    value = value * scale.repeat_interleave(16, dim=1)
    return value.reshape(gs.numel(), -1, value.shape[1]) * gs.double()[:, None, None]


def exact(case, seed):
    s = _inputs(case, seed)
    m, k = case["m"], case["top_k"]
    if case["op"] == "route":
        return _exact_route(case, s["logits"].double(), s["bias"])
    ids, x = s["ids"].long(), s["x"].double()
    if case["op"] == "linear":
        y = torch.zeros((m, k, case["n"]), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            i, j = torch.nonzero(ids == e, as_tuple=True)
            if i.numel():
                y[i, j] = x[i] @ _exact_weight(s["w"], e)[0].t()
        return y
    out = torch.zeros((m, case["hidden"]), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        i, j = torch.nonzero(ids == e, as_tuple=True)
        if i.numel():
            gate, up = (x[i] @ w.t() for w in _exact_weight(s["gate_up"], e))
            y = (gate * torch.sigmoid(gate) * up) @ _exact_weight(s["down"], e)[0].t()
            out.index_add_(0, i, s["weights"][i, j].double()[:, None] * y)
    return out


def _exact_route(case, logits, bias):
    m, e, k = case["m"], case["experts"], case["top_k"]
    if case["scoring"] == "softmax":
        score = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        score = score / score.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    key = score if bias is None else score + bias.double()
    key = key.masked_fill(logits == -math.inf, -math.inf)
    left = torch.ones((m, e), dtype=torch.bool, device="cuda")
    if case["groups"] > 1:
        size = e // case["groups"]
        first = key.reshape(m, -1, size).topk(min(2, size), dim=2).values
        first = torch.where((first == -math.inf) & (torch.arange(first.shape[2], device="cuda") > 0), 0.0, first)
        group = first.sum(dim=2) if case["group_score"] == "top2" else first[:, :, 0]
        left[:] = False
        for _ in range(case["top_groups"]):
            at = (group == group.amax(dim=1, keepdim=True)).int().argmax(dim=1)  # the lowest of equal ones
            left.view(m, -1, size)[torch.arange(m, device="cuda"), at] = group.gather(1, at[:, None]) > -math.inf
            group = group.scatter(1, at[:, None], -math.inf)
    ids, w = [], []
    for _ in range(k):
        open_ = torch.where(left, key, -math.inf)
        best = open_.amax(dim=1, keepdim=True)
        at = (open_ == best).int().argmax(dim=1, keepdim=True)
        there = best > -math.inf
        ids.append(torch.where(there, at, -1))
        w.append(torch.where(there, score.gather(1, at), 0.0))
        left.scatter_(1, at, False)
    ids, w = torch.cat(ids, dim=1), torch.cat(w, dim=1)
    if case["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    return {"ids": ids.to(torch.int32), "weights": case["scale"] * w}
