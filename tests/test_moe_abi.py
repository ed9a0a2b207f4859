"""Refusals of the mixture-of-experts entry points: every bad argument is an
error on the host, before anything touches the device."""
import ctypes

import pytest

from nvfp4_quantized_dense_w4a16_b200 import build as B

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 7


@pytest.fixture(scope="module")
def native():
    B.build()
    from nvfp4_quantized_dense_w4a16_b200 import native
    return native


FAKE = ctypes.c_void_p(256)


def route(native, m=4, experts=64, ld=None, type=0, logits=FAKE, ids=FAKE, weights=FAKE, bias=None, **kw):
    r = dict(scoring=0, top_k=8, groups=1, top_groups=1, group_score=0, renormalize=1, scale=1.0)
    r.update(kw)
    cfg = native.MoeRouter(**r)
    return native.lib.ffn_nvfp4_moe_route(logits, type, m, experts, experts if ld is None else ld, bias,
                                          ctypes.byref(cfg), ids, weights, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), INVALID), (dict(m=0), OK), (dict(m=0, logits=None, ids=None, weights=None), OK),
    (dict(type=2), INVALID), (dict(experts=0), INVALID), (dict(ld=63), INVALID),
    (dict(scoring=2), INVALID), (dict(group_score=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(top_k=0), INVALID), (dict(groups=0), INVALID),
    (dict(top_groups=0), INVALID), (dict(groups=2, top_groups=3), INVALID), (dict(groups=3), SHAPE),
    (dict(top_k=65, experts=64), SHAPE), (dict(groups=16, top_groups=1), SHAPE),
    (dict(top_k=33), UNSUPPORTED), (dict(experts=1025), UNSUPPORTED), (dict(groups=64, top_groups=64), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID),
    (dict(logits=ctypes.c_void_p(258)), ALIGN), (dict(logits=ctypes.c_void_p(257), type=1), ALIGN),
    (dict(ids=ctypes.c_void_p(258)), ALIGN), (dict(bias=ctypes.c_void_p(258)), ALIGN),
    (dict(m=1 << 31), SHAPE), (dict(m=1 << 28), SHAPE),
])
def test_route_refusals(native, kw, status):
    assert route(native, **kw) == status


def test_route_without_a_router(native):
    assert native.lib.ffn_nvfp4_moe_route(FAKE, 0, 4, 64, 64, None, None, FAKE, FAKE, None) == INVALID


@pytest.mark.parametrize("args,status", [
    ((None, FAKE, FAKE, 4, 64, 64, 0), INVALID), ((FAKE, None, FAKE, 4, 64, 64, 0), INVALID),
    ((FAKE, FAKE, None, 4, 64, 64, 0), INVALID), ((FAKE, FAKE, FAKE, 4, 64, 64, 2), INVALID),
    ((FAKE, FAKE, FAKE, 0, 64, 64, 0), SHAPE), ((FAKE, FAKE, FAKE, 4, 0, 64, 0), SHAPE),
    ((FAKE, FAKE, FAKE, 4, 64, 48, 0), SHAPE), ((FAKE, FAKE, FAKE, 4, 63, 64, 1), SHAPE),
    ((FAKE, FAKE, FAKE, 4, 96, 64, 1), SHAPE),  # inter = 48
    ((FAKE, FAKE, FAKE, 1025, 64, 64, 0), UNSUPPORTED),
    ((ctypes.c_void_p(264), FAKE, FAKE, 4, 64, 64, 0), ALIGN), ((FAKE, FAKE, ctypes.c_void_p(258), 4, 64, 64, 0), ALIGN),
])
def test_experts_create_refusals(native, args, status):
    h = ctypes.c_void_p()
    assert native.lib.ffn_nvfp4_experts_create(*args, None, ctypes.byref(h)) == status
    assert not h.value


def test_null_handles(native):
    L = native.lib
    assert L.ffn_nvfp4_experts_create(FAKE, FAKE, FAKE, 4, 64, 64, 0, None, None) == INVALID
    assert L.ffn_nvfp4_experts_destroy(None) == OK
    assert L.ffn_nvfp4_experts_info(None, None, None, None, None, None) == INVALID
    assert L.ffn_nvfp4_experts_linear(FAKE, 1, None, FAKE, 1, FAKE, FAKE, 1 << 20, None) == INVALID
    assert L.ffn_nvfp4_moe_forward(FAKE, 1, 64, 64, None, None, FAKE, FAKE, 1, FAKE, FAKE, 1 << 20, None) == INVALID


def test_workspace_sizes(native):
    L, out = native.lib, ctypes.c_size_t()
    size = lambda *a: native.ffn_nvfp4_moe_workspace_size(*a)
    assert size(0, 8, 64, 256, 512) == 0 and native.ffn_nvfp4_experts_workspace_size(0, 8, 64, 256, 512) == 0
    # the hidden rows and the experts' outputs of every (row, pick)
    assert size(37, 3, 20, 1056, 672) >= 37 * 3 * (672 * 2 + 1056 * 4)
    assert size(1, 1, 1, 32, 32) % 256 == 0
    for args, status in (((-1, 8, 64, 256, 512), INVALID), ((4, 0, 64, 256, 512), INVALID), ((4, 8, 0, 256, 512), INVALID),
                         ((4, 8, 64, 250, 512), SHAPE), ((4, 8, 64, 256, 500), SHAPE), ((1 << 28, 8, 64, 256, 512), SHAPE)):
        assert L.ffn_nvfp4_moe_workspace_size(*args, ctypes.byref(out)) == status, args
    assert L.ffn_nvfp4_moe_workspace_size(4, 8, 64, 256, 512, None) == INVALID
    for args, status in (((-1, 8, 64, 256, 512), INVALID), ((4, 8, 64, 0, 512), INVALID), ((4, 8, 64, 256, 500), SHAPE)):
        assert L.ffn_nvfp4_experts_workspace_size(*args, ctypes.byref(out)) == status, args


def test_sizes_that_overflow_are_refused(native):
    L, out = native.lib, ctypes.c_size_t()
    big = 1 << 40
    for args in ((1 << 24, 8, 64, 1 << 29, 512), (1, 1, 1, big, 32), (1, 1, 1, 32, big), (1 << 20, 32, 64, 1 << 18, 32),
                 (1, 1, 1, (1 << 63) - 32, 32)):
        assert L.ffn_nvfp4_moe_workspace_size(*args, ctypes.byref(out)) == SHAPE, args
        assert L.ffn_nvfp4_experts_workspace_size(*args, ctypes.byref(out)) == SHAPE, args
    for experts in (1025, 1 << 62):
        assert L.ffn_nvfp4_moe_workspace_size(1, 1, experts, 64, 64, ctypes.byref(out)) == UNSUPPORTED
        assert L.ffn_nvfp4_experts_workspace_size(1, 1, experts, 64, 64, ctypes.byref(out)) == UNSUPPORTED


@pytest.mark.parametrize("experts,top_k,hidden,inter", [
    (8, 2, 4096, 12288), (64, 8, 2048, 1024), (20, 3, 1056, 672), (1, 1, 32, 32), (3, 1, 256, 4096), (1024, 1, 64, 4096),
    (256, 8, 7168, 2048), (40, 33, 96, 1600), (2, 5, 128, 64),
])
def test_a_workspace_serves_every_smaller_batch(native, experts, top_k, hidden, inter):
    """A size never falls as m grows, where other kernels take over (32 pairs, 5 and 8 pairs an expert) or K is cut
    into fewer ranges as well."""
    last = 9 * max(32, 8 * experts) // top_k // 8 + 8
    layer = [native.ffn_nvfp4_moe_workspace_size(m, top_k, experts, hidden, inter) for m in range(last)]
    linear = [native.ffn_nvfp4_experts_workspace_size(m, top_k, experts, hidden, inter) for m in range(last)]
    for sizes in (layer, linear):
        falls = [(m, a, b) for m, (a, b) in enumerate(zip(sizes, sizes[1:])) if b < a]
        assert not falls, falls[:4]


@pytest.mark.parametrize("kw,name", [(dict(scoring="soft"), "scoring"), (dict(scoring=None), "scoring"),
                                     (dict(group_score="top3"), "group_score"), (dict(group_score=0), "group_score")])
def test_unknown_router_names_are_refused_by_name(native, kw, name):
    import torch
    with pytest.raises(ValueError, match=f"^{name} must be one of"):
        native.ffn_nvfp4_moe_route(torch.zeros((4, 32)), 4, **kw)
