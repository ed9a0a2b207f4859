"""What is measured of the 8-bit integer layers and of the norms around a layer, each with its plain form.

Three operators (a case's "op"):

* "norm":   what stands between two layers, in one call: z = norm(y) of a layer's output; r' = a * r + b * gate * z, the new
            residual, rounded to its type; x' = norm(r'), the next layer's input;
* "linear": y[i, j] = xs[i] * ws[j] * sum_k xq[i, k] * wq[j, k] (+ bias[j]) over int8 codes with a scale for each row (token) and
            each output channel; rows that come in bf16 are quantised first (scale = max |x| / 127);
* "ffn":    out = down(silu(gate(x)) * up(x)) of such products; the hidden rows are rounded to bf16 and quantised again.
            With "norms" the call stands in its block: norm and quantisation before it, norm, gate, residual and the next
            layer's norm after it.

Weights are drawn as codes of normal values with scales around one.  Activations have a few channels of larger values, and
tokens of differing size.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # between two layers of a decode step of one token: the latency of the call
        {"name": "norm one row", "op": "norm", "m": 1, "hidden": 4096, "residual": "bfloat16", "weight": "bfloat16", "kind": "rms", "offset": 0.0,
         "branch": True, "post": True, "pre": True, "gate": "none", "activation": "none", "residual_scale": 1.0, "branch_scale": 1.0},
        # a ragged decode batch of an odd width, layer norms, a gate for each token
        {"name": "norm ragged", "op": "norm", "m": 203, "hidden": 1037, "residual": "float32", "weight": "float32", "kind": "layer", "offset": 0.0,
         "branch": True, "post": False, "pre": True, "gate": "row", "activation": "sigmoid", "residual_scale": 1.0, "branch_scale": 1.0},
        # a prompt, norms before and after the layer, a gate for each channel, residual in fp32
        {"name": "norm prompt", "op": "norm", "m": 4096, "hidden": 5120, "residual": "float32", "weight": "bfloat16", "kind": "rms", "offset": 1.0,
         "branch": True, "post": True, "pre": True, "gate": "channel", "activation": "none", "residual_scale": 0.9, "branch_scale": 0.5},
        # long prompts of a narrow model, a gate for each value, residual in bf16
        {"name": "norm long prompt", "op": "norm", "m": 16384, "hidden": 2048, "residual": "bfloat16", "weight": "bfloat16", "kind": "rms", "offset": 0.0,
         "branch": True, "post": True, "pre": True, "gate": "full", "activation": "tanh", "residual_scale": 1.0, "branch_scale": 1.0},
        # one token through one projection
        {"name": "linear one row", "op": "linear", "m": 1, "n": 4096, "k": 4096, "bias": False, "quantized": False},
        # a ragged decode batch, sizes that are no multiple of a tile
        {"name": "linear ragged", "op": "linear", "m": 37, "n": 1000, "k": 1056, "bias": True, "quantized": False},
        # a short prompt through a deep projection, rows quantised before
        {"name": "linear 512 rows", "op": "linear", "m": 512, "n": 5120, "k": 17408, "bias": False, "quantized": True},
        # a prompt through a square projection
        {"name": "linear prompt", "op": "linear", "m": 4096, "n": 4096, "k": 4096, "bias": True, "quantized": False},
        # decode of one token
        {"name": "ffn one row", "op": "ffn", "m": 1, "hidden": 4096, "inter": 12288, "norms": False},
        # a decode batch in its block
        {"name": "block 48 rows", "op": "ffn", "m": 48, "hidden": 5120, "inter": 17408, "norms": True},
        # a ragged batch in its block
        {"name": "block ragged", "op": "ffn", "m": 301, "hidden": 1056, "inter": 672, "norms": True},
        # a prompt
        {"name": "ffn prompt", "op": "ffn", "m": 4096, "hidden": 4096, "inter": 12288, "norms": False},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over their logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "ffn", "ffn"])
    if op == "norm":
        while True:
            m, hidden = _log(rng, 1, 16384), rng.choice([_log(rng, 16, 8192), 8 * _log(rng, 8, 1024)])
            if m * hidden <= 32 * 10**6:
                break
        branch = rng.random() < 0.8
        post, pre = rng.choice([(True, True), (True, False), (False, True)]) if branch else (False, True)
        gate = rng.choice(["none", "row", "channel", "full"]) if branch else "none"
        return {"op": op, "m": m, "hidden": hidden, "residual": rng.choice(["bfloat16", "float32"]), "weight": rng.choice(["bfloat16", "float32"]),
                "kind": rng.choice(["rms", "rms", "layer"]), "offset": rng.choice([0.0, 1.0]), "branch": branch, "post": post, "pre": pre,
                "gate": gate, "activation": rng.choice(["none", "sigmoid", "tanh"]) if gate != "none" else "none",
                "residual_scale": rng.choice([1.0, 0.9]) if branch else 1.0, "branch_scale": rng.choice([1.0, 0.5]) if branch else 1.0}
    while True:
        case = {"op": op, "m": _log(rng, 1, 8192)}
        if op == "linear":
            case.update(n=_log(rng, 16, 16384), k=32 * _log(rng, 2, 544), bias=rng.random() < 0.5, quantized=rng.random() < 0.5)
            weights = case["n"] * case["k"]
        else:
            case.update(hidden=32 * _log(rng, 4, 192), inter=32 * _log(rng, 4, 544), norms=rng.random() < 0.5)
            weights = 3 * case["hidden"] * case["inter"]
        if weights <= 26 * 10**7 and 2 * case["m"] * weights <= 12 * 10**11:
            return case


# ------------------------------------------------------------------ inputs

def _rows(g, m, k):
    """Activations as a layer meets them: tokens of differing size, a few large channels."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x *= torch.exp(0.3 * torch.randn((m, 1), generator=g, device="cuda"))
    return x * torch.where(torch.rand((1, k), generator=g, device="cuda") < 0.01, 8.0, 1.0)


def _weight(g, n, k):
    """int8 codes [n, k] and the channels' scales [n]."""
    codes = torch.randn((n, k), generator=g, device="cuda").mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    scales = torch.exp(0.2 * torch.randn((n,), generator=g, device="cuda")) / (36.0 * math.sqrt(k))
    return codes, scales


def _norm(g, case):
    """A norm's weight (and bias)."""
    t = getattr(torch, case["weight"])
    w = 1.0 - case["offset"] + 0.2 * torch.randn((case["hidden"],), generator=g, device="cuda")
    bias = (0.1 * torch.randn((case["hidden"],), generator=g, device="cuda")).to(t) if case["kind"] == "layer" else None
    return w.to(t), bias


def _around(g, s, case):
    """A block's residual, gate and norms."""
    m, hidden = case["m"], case["hidden"]
    s["residual"] = (2.0 * _rows(g, m, hidden)).to(getattr(torch, case["residual"]))
    s["post"] = _norm(g, case) if case["post"] else None
    s["pre"] = _norm(g, case) if case["pre"] else None
    shape = {"none": None, "row": (m, 1), "channel": (1, hidden), "full": (m, hidden)}[case["gate"]]
    s["gate"] = None if shape is None else torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


#: The norms and the gate of an "ffn" case in its block.
_BLOCK = {"residual": "bfloat16", "weight": "bfloat16", "kind": "rms", "offset": 0.0, "branch": True, "post": True, "pre": True, "gate": "channel",
          "activation": "none", "residual_scale": 1.0, "branch_scale": 1.0}


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = case["m"]
    s = {"case": case}
    if case["op"] == "norm":
        _around(g, s, case)
        s["y"] = (0.5 * _rows(g, m, case["hidden"])).to(torch.bfloat16) if case["branch"] else None
        return s
    if case["op"] == "linear":
        x = _rows(g, m, case["k"]).to(torch.bfloat16)
        s["x"], s["x_scales"] = _codes(x) if case["quantized"] else (x, None)
        s["w"], s["w_scales"] = _weight(g, case["n"], case["k"])
        s["bias"] = torch.randn((case["n"],), generator=g, device="cuda").to(torch.bfloat16) if case["bias"] else None
        return s
    hidden, inter = case["hidden"], case["inter"]
    s["gate_up"], s["gate_up_scales"] = _weight(g, 2 * inter, hidden)
    s["down"], s["down_scales"] = _weight(g, hidden, inter)
    if case["norms"]:
        _around(g, s, {**case, **_BLOCK})
        s["first"] = _norm(g, {**case, **_BLOCK})
    else:
        s["x"] = _rows(g, m, hidden).to(torch.bfloat16)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from nvfp4_quantized_dense_w4a16_b200 import native as N
        empty = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
        m = case["m"]
        if case["op"] == "linear":
            s["out"] = empty((m, case["n"]), torch.bfloat16)
            size = N.ffn_int8_linear_workspace_size(m, case["n"], case["k"])
            s["workspace"] = empty((max(16, size),), torch.uint8)
            return s
        hidden = case["hidden"]
        for name in ("post", "pre", "first"):
            if s.get(name) is not None:
                kind, offset = (case["kind"], case["offset"]) if case["op"] == "norm" else (_BLOCK["kind"], _BLOCK["offset"])
                s[name] = N.Norm(s[name][0], s[name][1], kind=kind, offset=offset)
        if case["op"] == "ffn":
            s["out"] = empty((m, hidden), torch.bfloat16)
            size = N.ffn_int8_workspace_size(m, hidden, case["inter"])
            s["workspace"] = empty((max(16, size),), torch.uint8)
            if not case["norms"]:
                return s
            s["codes"], s["scales"] = empty((m, hidden), torch.int8), empty((m,), torch.float32)
        s["residual_out"] = torch.empty_like(s["residual"]) if case.get("branch", True) else None
        s["next"] = empty((m, hidden), torch.bfloat16) if s["pre"] is not None else None
    return s


# ------------------------------------------------------------------ plain forms

def _codes(x):
    """int8 codes and fp32 scales of bf16 rows."""
    x = x.float()
    top = x.abs().amax(dim=1, keepdim=True)
    codes = torch.where(top > 0, torch.round(x * (127.0 / top)), 0.0)
    return codes.to(torch.int8), (top / 127.0)[:, 0]


def _product(x, x_scales, w, w_scales):
    y = x.float() @ w.float().t()
    return y * x_scales[:, None] * w_scales


def _plain_ffn(x, x_scales, s):
    gate, up = _product(x, x_scales, s["gate_up"], s["gate_up_scales"]).chunk(2, dim=1)
    h = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)
    return _product(*_codes(h), s["down"], s["down_scales"]).to(torch.bfloat16)


def _plain_norm(x, weights, case):
    w, bias = weights
    if case["kind"] == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(dim=1, keepdim=True) + 1e-6) * (w.float() + case["offset"])
    return x if bias is None else x + bias.float()


def _plain_around(y, s, case):
    r = s["residual"]
    if y is not None:
        z = y.float()
        if s["post"] is not None:
            z = _plain_norm(z, s["post"], case)
        if s["gate"] is not None:
            gate = s["gate"].float()
            gate = 1.0 / (1.0 + torch.exp(-gate)) if case["activation"] == "sigmoid" else torch.tanh(gate) if case["activation"] == "tanh" else gate
            z = z * gate
        r = (case["residual_scale"] * r.float() + case["branch_scale"] * z).to(r.dtype)
    out = {"residual": r} if y is not None else {}
    if s["pre"] is not None:
        out["x"] = _plain_norm(r.float(), s["pre"], case).to(torch.bfloat16)
    return out


def run(s):
    c = s["case"]
    if own:
        from nvfp4_quantized_dense_w4a16_b200 import native as N
        if c["op"] == "linear":
            return N.ffn_int8_linear(s["x"], s["w"], s["w_scales"], x_scales=s["x_scales"], bias=s["bias"], y=s["out"], workspace=s["workspace"])
        if c["op"] == "ffn":
            x, x_scales = (s["x"], None) if not c["norms"] else N.ffn_block_norm(
                s["residual"], pre=s["first"], quantize=True, out=s["codes"], out_scales=s["scales"])[1:]
            y = N.ffn_int8_forward(x, s["gate_up"], s["gate_up_scales"], s["down"], s["down_scales"], x_scales=x_scales, out=s["out"],
                                   workspace=s["workspace"])
            if not c["norms"]:
                return y
            c = _BLOCK
        else:
            y = s["y"]
        r, x = N.ffn_block_norm(s["residual"], y=y, post=s["post"], gate=s["gate"], gate_activation=c["activation"],
                                residual_scale=c["residual_scale"], branch_scale=c["branch_scale"], pre=s["pre"],
                                residual_out=s["residual_out"], out=s["next"])
        out = {"residual": r} if y is not None else {}
        return out if x is None else {**out, "x": x}
    if c["op"] == "norm":
        return _plain_around(s["y"], s, c)
    if c["op"] == "linear":
        x, x_scales = (s["x"], s["x_scales"]) if c["quantized"] else _codes(s["x"])
        y = _product(x, x_scales, s["w"], s["w_scales"])
        return (y if s["bias"] is None else y + s["bias"].float()).to(torch.bfloat16)
    if not c["norms"]:
        return _plain_ffn(*_codes(s["x"]), s)
    x = _plain_norm(s["residual"].float(), s["first"], _BLOCK).to(torch.bfloat16)
    return _plain_around(_plain_ffn(*_codes(x), s), s, _BLOCK)


# ------------------------------------------------------------------ floors and exact values

def work(case):
    m = case["m"]
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        x = m * k + 4 * m if case["quantized"] else 2 * m * k
        return {"bytes": n * k + 4 * n + x + 2 * n * case["bias"] + 2 * m * n, "flops": 2 * m * n * k}
    hidden, bytes_, flops = case["hidden"], 0, 0
    if case["op"] == "ffn":
        weights = 3 * hidden * case["inter"]
        bytes_, flops = weights + 4 * (2 * case["inter"] + hidden), 2 * m * weights
        if not case["norms"]:
            return {"bytes": bytes_ + 4 * m * hidden, "flops": flops}
        case = {**case, **_BLOCK}
        bytes_ -= 2 * m * hidden  # (the layer's output need not leave the chip)
    size = 2 if case["residual"] == "bfloat16" else 4
    gate = {"none": 0, "row": m, "channel": hidden, "full": m * hidden}[case["gate"]]
    norms = (case["post"] + case["pre"]) * (2 if case["kind"] == "layer" else 1) * (2 if case["weight"] == "bfloat16" else 4) * hidden
    bytes_ += m * hidden * (size + (size + 2) * case["branch"] + 2 * case["pre"]) + 2 * gate + norms
    return {"bytes": bytes_, "flops": flops + 16 * m * hidden}


def _exact_codes(x):
    """Whole numbers in 64 bits, and scales, of rows: the nearest multiples of max |x| / 127."""
    x = x.double()
    step = x.abs().max(dim=1).values / 127.0
    return torch.round(x / step.clamp(min=1e-300)[:, None]), step


def _exact_product(codes, scales, w, w_scales):
    """In pieces of the channels; the sums are whole numbers below 2^53."""
    parts = [torch.mm(codes, part.double().t()) * s.double() for part, s in zip(w.split(4096), w_scales.split(4096))]
    return torch.cat(parts, dim=1) * scales.double()[:, None]


def _exact_norm(v, weights, case):
    v = v.double()
    mean = v.sum(dim=1, keepdim=True) / v.shape[1] if case["kind"] == "layer" else torch.zeros_like(v[:, :1])
    v = v - mean
    v = v / torch.sqrt((v * v).sum(dim=1, keepdim=True) / v.shape[1] + 1e-6) * (weights[0].double() + case["offset"])
    return v if weights[1] is None else v + weights[1].double()


def _exact_around(y, s, case):
    r, out = s["residual"].double(), {}
    if y is not None:
        z = _exact_norm(y, s["post"], case) if s["post"] is not None else y.double()
        if s["gate"] is not None:
            gate = s["gate"].double()
            z = z * {"none": lambda t: t, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[case["activation"]](gate)
        r = out["residual"] = case["residual_scale"] * r + case["branch_scale"] * z
    if s["pre"] is not None:
        out["x"] = _exact_norm(r.to(s["residual"].dtype), s["pre"], case)  # (of the residual as it is stored)
    return out


def _exact_ffn(codes, scales, s):
    gate, up = _exact_product(codes, scales, s["gate_up"], s["gate_up_scales"]).chunk(2, dim=1)
    h = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16)
    return _exact_product(*_exact_codes(h), s["down"], s["down_scales"])


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm":
        return _exact_around(s["y"], s, case)
    if case["op"] == "linear":
        codes, scales = (s["x"].double(), s["x_scales"]) if case["quantized"] else _exact_codes(s["x"])
        y = _exact_product(codes, scales, s["w"], s["w_scales"])
        return y if s["bias"] is None else y + s["bias"].double()
    if not case["norms"]:
        return _exact_ffn(*_exact_codes(s["x"]), s)
    x = _exact_norm(s["residual"], s["first"], _BLOCK).to(torch.bfloat16)
    return _exact_around(_exact_ffn(*_exact_codes(x), s).to(torch.bfloat16), s, _BLOCK)
