"""Refusals of the 8-bit integer entry points and of ffn_block_norm: every bad
argument is an error on the host, before anything touches the device."""
import ctypes

import pytest

from nvfp4_quantized_dense_w4a16_b200 import build as B

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 7


@pytest.fixture(scope="module")
def native():
    B.build()
    from nvfp4_quantized_dense_w4a16_b200 import native
    return native


def at(address):
    return ctypes.c_void_p(address)


FAKE = at(256)


@pytest.mark.parametrize("args,status", [
    ((FAKE, -1, 64, 64, FAKE, FAKE), INVALID), ((FAKE, 0, 64, 64, FAKE, FAKE), OK), ((None, 0, 64, 64, None, None), OK),
    ((FAKE, 4, 0, 64, FAKE, FAKE), SHAPE), ((FAKE, 4, 48, 64, FAKE, FAKE), SHAPE), ((FAKE, 4, 64, 63, FAKE, FAKE), INVALID),
    ((FAKE, 4, 64, 68, FAKE, FAKE), ALIGN), ((at(264), 4, 64, 64, FAKE, FAKE), ALIGN), ((FAKE, 4, 64, 64, at(264), FAKE), ALIGN),
    ((FAKE, 4, 64, 64, FAKE, at(258)), ALIGN), ((None, 4, 64, 64, FAKE, FAKE), INVALID), ((FAKE, 4, 64, 64, None, FAKE), INVALID),
    ((FAKE, 4, 64, 64, FAKE, None), INVALID), ((FAKE, 1 << 30, 1 << 20, 1 << 20, FAKE, FAKE), SHAPE),
    ((FAKE, 1 << 31, 64, 64, FAKE, FAKE), SHAPE),
])
def test_quantize_refusals(native, args, status):
    assert native.lib.ffn_int8_quantize(*args, None) == status


def linear(native, x=FAKE, xs=FAKE, m=4, w=FAKE, ws=FAKE, bias=None, n=64, k=64, y=FAKE, work=FAKE, size=1 << 20):
    return native.lib.ffn_int8_linear(x, xs, m, w, ws, bias, n, k, y, work, size, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), INVALID), (dict(m=0), OK), (dict(m=0, x=None, y=None, work=None), OK), (dict(n=0), SHAPE), (dict(k=0), SHAPE),
    (dict(k=48), SHAPE), (dict(k=131072), UNSUPPORTED), (dict(m=1 << 31), SHAPE), (dict(m=1 << 29, n=1 << 12), SHAPE),
    (dict(n=1 << 29, k=1 << 12), SHAPE), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(ws=None), INVALID),
    (dict(y=None), INVALID), (dict(xs=None, work=None), WORKSPACE), (dict(xs=None, size=255), WORKSPACE),
    (dict(x=at(264)), ALIGN), (dict(w=at(264)), ALIGN), (dict(y=at(264)), ALIGN), (dict(ws=at(258)), ALIGN),
    (dict(xs=at(258)), ALIGN), (dict(bias=at(257)), ALIGN), (dict(xs=None, work=at(264)), ALIGN),
])
def test_linear_refusals(native, kw, status):
    assert linear(native, **kw) == status


def forward(native, x=FAKE, xs=FAKE, m=4, hidden=64, inter=96, gu=FAKE, gus=FAKE, dn=FAKE, dns=FAKE, out=FAKE, work=FAKE,
            size=1 << 20):
    return native.lib.ffn_int8_forward(x, xs, m, hidden, inter, gu, gus, dn, dns, out, work, size, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), INVALID), (dict(m=0), OK), (dict(m=0, x=None, out=None, work=None), OK), (dict(hidden=0), SHAPE),
    (dict(hidden=48), SHAPE), (dict(inter=0), SHAPE), (dict(inter=100), SHAPE), (dict(hidden=131072), UNSUPPORTED),
    (dict(inter=131072), UNSUPPORTED), (dict(m=1 << 31), SHAPE), (dict(x=None), INVALID), (dict(gu=None), INVALID),
    (dict(gus=None), INVALID), (dict(dn=None), INVALID), (dict(dns=None), INVALID), (dict(out=None), INVALID),
    (dict(work=None), WORKSPACE), (dict(size=255), WORKSPACE), (dict(x=at(264)), ALIGN), (dict(gu=at(264)), ALIGN),
    (dict(gus=at(258)), ALIGN), (dict(dn=at(264)), ALIGN), (dict(dns=at(258)), ALIGN), (dict(out=at(264)), ALIGN),
    (dict(work=at(264)), ALIGN), (dict(xs=at(258)), ALIGN),
])
def test_forward_refusals(native, kw, status):
    assert forward(native, **kw) == status


def test_workspace_sizes(native):
    L, out = native.lib, ctypes.c_size_t()
    assert native.ffn_int8_linear_workspace_size(0, 5, 64) == 0 and native.ffn_int8_workspace_size(0, 64, 96) == 0
    assert native.ffn_int8_linear_workspace_size(7, 5, 1056) >= 7 * 1056 + 28
    assert native.ffn_int8_workspace_size(7, 1056, 672) >= 7 * (1056 + 3 * 672 + 8)
    for m in range(1, 600):  # a size serves every smaller batch
        assert native.ffn_int8_linear_workspace_size(m, 1000, 1056) >= native.ffn_int8_linear_workspace_size(m - 1, 1000, 1056)
        assert native.ffn_int8_workspace_size(m, 1056, 672) >= native.ffn_int8_workspace_size(m - 1, 1056, 672)
    assert L.ffn_int8_linear_workspace_size(1, 1, 64, None) == INVALID and L.ffn_int8_workspace_size(1, 64, 64, None) == INVALID
    for args, status in (((-1, 1, 64), INVALID), ((1, 0, 64), SHAPE), ((1, 1, 65), SHAPE), ((1, 1, 1 << 20), UNSUPPORTED),
                         ((1 << 30, 1, 1 << 15), SHAPE), ((1, 1 << 62, 64), SHAPE), ((1 << 62, 1, 64), SHAPE)):
        assert L.ffn_int8_linear_workspace_size(*args, ctypes.byref(out)) == status, args
    for args, status in (((-1, 64, 64), INVALID), ((1, 64, 65), SHAPE), ((1, 1 << 20, 64), UNSUPPORTED), ((1 << 30, 64, 1 << 15), SHAPE)):
        assert L.ffn_int8_workspace_size(*args, ctypes.byref(out)) == status, args


class BlockArgs(ctypes.Structure):
    _fields_ = [("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64), ("post", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("gate_type", ctypes.c_int), ("gate_activation", ctypes.c_int), ("gate_row_stride", ctypes.c_int64),
                ("gate_col_stride", ctypes.c_int64), ("residual", ctypes.c_void_p), ("residual_type", ctypes.c_int),
                ("residual_stride", ctypes.c_int64), ("residual_out", ctypes.c_void_p), ("residual_out_stride", ctypes.c_int64),
                ("residual_scale", ctypes.c_float), ("branch_scale", ctypes.c_float), ("pre", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64), ("out_scales", ctypes.c_void_p)]


def block(native, m=4, hidden=64, norm={}, **kw):
    n = native._NormStruct(**{"kind": 0, "type": 1, "weight": 256, "bias": None, "eps": 1e-6, "offset": 0.0, **norm})
    a = dict(y=256, y_stride=64, post=ctypes.addressof(n), gate=256, gate_type=1, gate_activation=1, gate_row_stride=64,
             gate_col_stride=1, residual=256, residual_type=1, residual_stride=64, residual_out=256, residual_out_stride=64,
             residual_scale=1.0, branch_scale=1.0, pre=ctypes.addressof(n), out=256, out_stride=64, out_scales=None)
    a.update(kw)
    return native.lib.ffn_block_norm(ctypes.byref(BlockArgs(**a)), m, hidden, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(m=0), OK), (dict(m=0, residual=None, out=None), OK), (dict(m=-1), INVALID), (dict(hidden=0), INVALID),
    (dict(residual_type=2), INVALID), (dict(residual_scale=NAN), INVALID), (dict(branch_scale=INF), INVALID),
    (dict(norm=dict(kind=2)), INVALID), (dict(norm=dict(type=-1)), INVALID), (dict(norm=dict(eps=0.0)), INVALID),
    (dict(norm=dict(eps=-1.0)), INVALID), (dict(norm=dict(eps=NAN)), INVALID), (dict(norm=dict(eps=INF)), INVALID),
    (dict(norm=dict(offset=NAN)), INVALID), (dict(gate_type=3), INVALID), (dict(gate_activation=3), INVALID),
    (dict(gate_col_stride=2), INVALID), (dict(gate_row_stride=-1), INVALID), (dict(gate_row_stride=63), INVALID),
    (dict(y=None), INVALID), (dict(y=None, post=None), INVALID), (dict(y=None, post=None, gate=None), INVALID),
    (dict(y=None, post=None, gate=None, residual_out=None, residual_scale=0.5), INVALID),
    (dict(y=None, post=None, gate=None, residual_out=None, pre=None, out=None), INVALID),
    (dict(pre=None), INVALID), (dict(pre=None, out=None, out_scales=256), INVALID), (dict(residual=None), INVALID),
    (dict(out=None), INVALID), (dict(pre=None, out=None, residual_out=None), INVALID),
    (dict(y_stride=63), INVALID), (dict(residual_stride=63), INVALID), (dict(residual_out_stride=63), INVALID),
    (dict(out_stride=63), INVALID),
    (dict(hidden=32776, y_stride=40000, residual_stride=40000, residual_out_stride=40000, out_stride=40000, gate_row_stride=0), UNSUPPORTED),
    (dict(out_scales=256, out_stride=72), SHAPE), (dict(out_scales=256, hidden=48, out_stride=48), SHAPE),
    (dict(m=1 << 40), SHAPE), (dict(m=1 << 62), SHAPE), (dict(residual_stride=1 << 40), SHAPE), (dict(gate_row_stride=1 << 40), SHAPE),
    (dict(y=257), ALIGN), (dict(residual=257), ALIGN), (dict(residual=258, residual_type=0), ALIGN), (dict(residual_out=257), ALIGN),
    (dict(out=257), ALIGN), (dict(gate=257), ALIGN), (dict(gate=258, gate_type=0), ALIGN), (dict(out_scales=258), ALIGN),
    (dict(norm=dict(weight=257)), ALIGN), (dict(norm=dict(bias=258, type=0)), ALIGN),
])
def test_block_norm_refusals(native, kw, status):
    assert block(native, **kw) == status


def test_block_norm_without_arguments(native):
    assert native.lib.ffn_block_norm(None, 4, 64, None) == INVALID


def test_python_refusals(native):
    import torch
    x, c, s = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    for call in (lambda: native.ffn_int8_quantize(x), lambda: native.ffn_int8_linear(x, c, s), lambda: native.ffn_int8_linear(c, c, s, x_scales=s),
                 lambda: native.ffn_int8_forward(x, c, s, c, s), lambda: native.ffn_block_norm(x), lambda: native.Norm(s)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        native.ffn_int8_quantize([1.0])
    with pytest.raises(ValueError, match="^kind must be one of"):
        native.Norm(kind="batch")
