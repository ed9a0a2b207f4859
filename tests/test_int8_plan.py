"""The choice of the 8-bit integer layers' kernels, host side: every kernel, tile
width and cut of K that layers of real sizes take is one that the GPU tests run."""
import ctypes

import pytest
import torch

from nvfp4_quantized_dense_w4a16_b200 import build as B
import test_gpu_int8_kernels as K

OK, INVALID, SHAPE, UNSUPPORTED = 0, 1, 2, 4


@pytest.fixture(scope="module")
def native():
    B.build()
    from nvfp4_quantized_dense_w4a16_b200 import native
    return native


@pytest.mark.parametrize("args,status", [
    ((4, 64, 64, 0), OK), ((0, 64, 64, 0), OK), ((4, 64, 64, 1), OK), ((4, 64, 64, 2), OK), ((-1, 64, 64, 0), INVALID), ((4, 64, 64, 3), INVALID),
    ((4, 64, 64, -1), INVALID), ((4, 0, 64, 0), SHAPE), ((4, 64, 48, 0), SHAPE), ((4, 65, 64, 0), OK), ((4, 65, 64, 1), SHAPE),
    ((4, 64, 131072, 0), UNSUPPORTED), ((1 << 31, 64, 64, 0), SHAPE)])
def test_refusals(native, args, status):
    p = native.Int8Plan()
    assert native.lib.ffn_int8_projection_plan(*args, ctypes.byref(p)) == status
    assert native.lib.ffn_int8_projection_plan(*args, None) == INVALID


def test_no_rows_take_no_kernel(native):
    assert native.ffn_int8_projection_plan(0, 64, 64) == {"kernel": "none", "tile_rows": 0, "tile_columns": 0, "k_splits": 0, "grid": 0, "turns": 0}


needs_148_sms = pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 148,
                                   reason="the cases are those of 148 SMs")


@needs_148_sms
def test_what_the_gpu_tests_run(native):
    plan = native.ffn_int8_projection_plan
    cut = set()
    for m, hidden, inter in K.CLUSTERS:
        p = plan(m, 2 * inter, hidden, "gate_up")
        assert p["kernel"] == "clusters"
        cut.add((p["k_splits"], -(-m // 128)))
    assert {c for c, _ in cut} >= {1, 5, 6, 8} and {b for _, b in cut} == {1, 2, 3, 4}
    for cases, role in ((K.PAIRS, "linear"), (K.GATE_UP_PAIRS, "gate_up")):
        seen = set()
        for m, a, b, columns, turns in cases:
            p = plan(m, a, b) if role == "linear" else plan(m, 2 * b, a, role)
            assert (p["kernel"], p["tile_columns"]) == ("pairs", columns) and p["turns"] >= turns
            seen.add((columns, turns >= 3))
        assert {c for c, _ in seen} == set(range(64, 257, 32)) and (256, True) in seen


@needs_148_sms
def test_what_layers_of_real_sizes_take(native):
    """A change of the estimates that sends these elsewhere asks for other cases in the GPU tests."""
    plan = native.ffn_int8_projection_plan
    for hidden, inter in ((4096, 12288), (5120, 17408), (7168, 2048)):
        assert plan(1, 2 * inter, hidden, "gate_up")["kernel"] == "row"
        for m in (2, 16, 48, 128):
            assert plan(m, 2 * inter, hidden, "gate_up")["kernel"] == "clusters"
        p = plan(4096, 2 * inter, hidden, "gate_up")
        assert p["kernel"] == "pairs" and p["turns"] >= 3
    assert plan(1, 2 * 28672, 8192, "gate_up")["turns"] == 2
