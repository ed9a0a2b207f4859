"""native.Norm hands each call its tensors and numbers as they are then (host
side; vectors on the CPU stand for device vectors, nothing is launched)."""
import pytest
import torch

from nvfp4_quantized_dense_w4a16_b200 import build as B


@pytest.fixture
def native(monkeypatch):
    B.build()
    from nvfp4_quantized_dense_w4a16_b200 import native

    def need(t, name, dtype, shape=None):
        if t.dtype is not dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dtype}")

    monkeypatch.setattr(native, "_need", need)
    return native


def bound(native, norm, hidden=64):
    now = native._norm_now(norm, "pre", hidden, -1)
    s = native._NormStruct.from_address(now[0])
    return s.weight, s.bias, s.type, s.kind, s.eps, s.offset


def test_storage_that_is_swapped_is_read_where_it_is(native):
    w, b = torch.nn.Parameter(torch.ones(64)), torch.zeros(64)
    n = native.Norm(w, b, kind="layer")
    assert bound(native, n)[:4] == (w.data_ptr(), b.data_ptr(), 0, 1)
    w.data = torch.full((64,), 2.0)
    b.set_(torch.ones(64))
    assert bound(native, n)[:2] == (w.data_ptr(), b.data_ptr())
    n = native.Norm(w)
    w.data = w.data.to(torch.bfloat16)  # (a module's `to` on the same Parameter)
    assert bound(native, n)[:4] == (w.data_ptr(), None, 1, 0)
    w.data = torch.ones(32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="32 weights, the rows 64"):
        bound(native, n)
    assert bound(native, n, 32)[0] == w.data_ptr() and n.hidden == 32
    w.data = torch.ones(64)[::2]
    with pytest.raises(ValueError, match="contiguous"):
        bound(native, n, 32)
    w.data = torch.ones(64, dtype=torch.float64)
    with pytest.raises(ValueError):
        bound(native, n)
    w.data = torch.ones(64)
    w.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="no storage"):
        bound(native, n)


def test_attributes_that_are_set_hold_from_the_next_call_on(native):
    w, other = torch.ones(64), torch.full((64,), 2.0)
    n = native.Norm(w)
    n.weight, n.eps, n.offset, n.kind = other, 1e-5, 1.0, "layer"
    assert bound(native, n) == (other.data_ptr(), None, 0, 1, pytest.approx(1e-5), 1.0)
    n.bias = w
    assert bound(native, n)[:2] == (other.data_ptr(), w.data_ptr())
    for name, value in (("bias", torch.ones(32)), ("weight", torch.ones(64, dtype=torch.bfloat16)), ("kind", "batch")):
        with pytest.raises(ValueError):
            setattr(n, name, value)
    assert bound(native, n)[:4] == (other.data_ptr(), w.data_ptr(), 0, 1) and n.bias is w and n.kind == "layer"
    n.bias = None
    n.weight = None
    assert bound(native, n, 7)[:2] == (None, None)
    for name in ("hidden", "device_index"):
        with pytest.raises(AttributeError):
            setattr(n, name, 3)
    n.name = "before the first layer"  # (a caller's own)
    assert n.name == "before the first layer"


def test_a_call_keeps_the_struct_that_it_was_given(native):
    """Another thread may swap the weight between a call's arguments and its launch."""
    w = torch.nn.Parameter(torch.ones(64))
    n = native.Norm(w)
    now = native._norm_now(n, "pre", 64, -1)
    before = w.data
    w.data = torch.zeros(64)
    then = native._norm_now(n, "pre", 64, -1)
    assert then[0] != now[0] and native._NormStruct.from_address(now[0]).weight == before.data_ptr()
    assert native._NormStruct.from_address(then[0]).weight == w.data_ptr()
