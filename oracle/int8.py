"""Plain numpy 8-bit integer layers and norms around a layer.  Test
infrastructure only.

Every step is written from the definitions in include/ffn_nvfp4.h; nothing here
is shared with the library.  Steps that the definitions fix to fp32 operations
are done in numpy's float32 (IEEE, each operation rounded once), so that they can
be compared bit for bit; norms are in fp64.
"""
from __future__ import annotations

import numpy as np

from . import nvfp4_ffn as O

F = np.float32


def quantize_rows(x):
    """(codes int8, scales float32) of rows of bf16 values given in any float type."""
    x = np.asarray(x, dtype=F)
    codes, scales = np.zeros(x.shape, np.int8), np.zeros(x.shape[0], F)
    for i, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            scales[i] = np.nan
            continue
        a = F(np.max(np.abs(row)))
        scales[i] = a / F(127)
        if a > 0:
            pre = F(2.0 ** 64) if a < F(2.0 ** -100) else F(1)
            codes[i] = np.rint((row * pre) * (F(127) / (a * pre))).astype(np.int8)
    return codes, scales


def sums(xq, wq):
    """Exact whole-number sums [m, n] (int64)."""
    y = np.zeros((xq.shape[0], wq.shape[0]), np.int64)
    for k in range(0, xq.shape[1], 8192):  # whole numbers below 2^53: products in float64 are exact
        y += (xq[:, k:k + 8192].astype(np.float64) @ wq[:, k:k + 8192].astype(np.float64).T).astype(np.int64)
    return y


def scaled(s, xs, ws):
    """float32 (sum * xs) * ws, each operation rounded once."""
    with np.errstate(invalid="ignore", over="ignore"):
        return (s.astype(F) * xs[:, None].astype(F)) * ws[None, :].astype(F)


def linear(xq, xs, wq, ws, bias=None):
    """y before its rounding to bf16, float32, bit for bit; bias: bf16 values."""
    v = scaled(sums(xq, wq), xs, ws)
    return v if bias is None else v + np.asarray(bias, dtype=F)[None, :]


def hidden_rows(xq, xs, gate_up, gate_up_scales):
    """(gate, h) in fp64 from the fp32 products' definition; h before its rounding to bf16."""
    inter = gate_up.shape[0] // 2
    s = sums(xq, gate_up).astype(np.float64)
    v = s * xs[:, None].astype(np.float64) * gate_up_scales[None, :].astype(np.float64)
    g, u = v[:, :inter], v[:, inter:]
    with np.errstate(over="ignore"):
        return g, g / (1.0 + np.exp(-g)) * u


def forward(xq, xs, gate_up, gate_up_scales, down, down_scales):
    """out before its rounding to bf16, float32."""
    h = O.round_to_bf16(hidden_rows(xq, xs, gate_up, gate_up_scales)[1])
    return linear(*quantize_rows(h), down, down_scales)


def norm(v, weight=None, bias=None, kind="rms", eps=1e-6, offset=0.0):
    """fp64, rows."""
    v = np.asarray(v, dtype=np.float64)
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    v = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    if weight is not None:
        v = v * (offset + np.asarray(weight, dtype=np.float64))
    return v if bias is None else v + np.asarray(bias, dtype=np.float64)


def gate_value(g, activation):
    g = np.asarray(g, dtype=np.float64)
    if activation == "sigmoid":
        return 1.0 / (1.0 + np.exp(-g))
    return np.tanh(g) if activation == "tanh" else g


def residual(r, z, gate=None, activation="none", residual_scale=1.0, branch_scale=1.0):
    """fp64 residual_scale * r + branch_scale * act(gate) * z."""
    g = 1.0 if gate is None else gate_value(gate, activation)
    return float(F(residual_scale)) * np.asarray(r, dtype=np.float64) + float(F(branch_scale)) * (g * np.asarray(z, dtype=np.float64))
