"""Plain numpy fp64 mixture of experts over NVFP4 weights: routing, products
by expert, the experts' SwiGLU layer.  Test infrastructure only.

Every step is written from the definitions in include/ffn_nvfp4.h, one row (or
one expert) at a time; nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np

from . import nvfp4_ffn as O


def log_score(logits: np.ndarray, scoring: str) -> np.ndarray:
    """log softmax / log sigmoid of finite or -inf logits, fp64."""
    l = np.asarray(logits, dtype=np.float64)
    if scoring == "softmax":
        top = l.max()
        with np.errstate(invalid="ignore"):
            return (l - top) - np.log(np.exp(l - top).sum())  # (top + log would swallow the log of huge logits)
    with np.errstate(over="ignore"):
        return np.where(l < 0, l - np.log1p(np.exp(np.minimum(l, 0))), -np.log1p(np.exp(-np.maximum(l, 0))))


def route_row(logits, bias, top_k, scoring="softmax", groups=1, top_groups=1, group_score="max", renormalize=True,
              scale=1.0):
    """(ids, weights) of one row; the row has no NaN (and no +inf under softmax)."""
    l = np.asarray(logits, dtype=np.float64)
    n = l.size
    ls = log_score(l, scoring) if np.any(l > -np.inf) else np.full(n, -np.inf)
    key = np.exp(ls) + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
    key = np.where((l > -np.inf) & (key > -np.inf), key, -np.inf)

    def place(e):  # the experts' order: key, logit (where the key is finite), id
        return -key[e], -l[e] if np.isfinite(key[e]) else 0.0, e

    if groups > 1:
        size = n // groups
        scores = []
        for g in range(groups):
            best = sorted((e for e in range(g * size, (g + 1) * size) if key[e] > -np.inf), key=place)
            if not best:
                scores.append((np.inf, 0.0, g))
            elif group_score == "top2":
                scores.append((-key[best[:2]].sum(), 0.0, g))
            else:
                scores.append(place(best[0]))
        open_ = sorted(range(groups), key=lambda g: scores[g])[:top_groups]
        key = np.where(np.isin(np.arange(n) // size, open_), key, -np.inf)
    order = sorted((e for e in range(n) if key[e] > -np.inf), key=place)[:top_k]
    ids = np.full(top_k, -1, dtype=np.int32)
    w = np.zeros(top_k)
    ids[:len(order)] = order
    if order:
        s = ls[order]
        if renormalize:
            s = np.exp(s - s.max())
            s = s / s.sum()
        else:
            s = np.exp(s)
        w[:len(order)] = scale * s
    return ids, w


def route(logits, bias, top_k, **kw):
    rows = [route_row(r, bias, top_k, **kw) for r in np.asarray(logits)]
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def experts_dequant(codes, block_scales, global_scales) -> np.ndarray:
    """fp64 weights [E, n, k]; global_scales [E], or [E, 2] for gate and up rows."""
    gs = np.asarray(global_scales, dtype=np.float64).reshape(codes.shape[0], -1)
    n = codes.shape[1]
    w = np.stack([O.dequantize(c, s) for c, s in zip(codes, block_scales)]).astype(np.float64)
    return w * np.repeat(gs, n // gs.shape[1], axis=1)[:, :, None]


def experts_linear(x, w, ids) -> np.ndarray:
    """fp64 y [m, top_k, n], unrounded; x [m, k] fp64, w [E, n, k] fp64."""
    m, top_k = ids.shape
    y = np.zeros((m, top_k, w.shape[1]))
    for i in range(m):
        for j in range(top_k):
            if 0 <= ids[i, j] < w.shape[0]:
                y[i, j] = w[ids[i, j]] @ x[i]
    return y


def moe_hidden(x, w_gate_up, ids):
    """Unrounded gate and up products and h = silu(gate) * up rounded to bf16, each [m, top_k, inter]."""
    gu = experts_linear(x, w_gate_up, ids)
    inter = gu.shape[2] // 2
    g, u = gu[:, :, :inter], gu[:, :, inter:]
    with np.errstate(over="ignore"):
        h = O.round_to_bf16(g / (1.0 + np.exp(-g)) * u)
    return g, u, np.asarray(h, dtype=np.float64)


def moe_forward(x, w_gate_up, w_down, ids, weights) -> np.ndarray:
    """fp64 out [m, hidden], unrounded."""
    h = moe_hidden(x, w_gate_up, ids)[2]
    out = np.zeros((x.shape[0], w_down.shape[1]))
    for j in range(ids.shape[1]):
        y = np.stack([w_down[e] @ h[i, j] if 0 <= e < w_down.shape[0] else np.zeros(w_down.shape[1])
                      for i, e in enumerate(ids[:, j])])
        out += np.asarray(weights, dtype=np.float64)[:, j, None] * y
    return out
