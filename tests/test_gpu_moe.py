"""Mixture of experts on the GPU against the fp64 oracle: routing decisions and
weights, products by expert, the layer, and the three of them together."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import moe as M
from oracle import nvfp4_ffn as O
from nvfp4_quantized_dense_w4a16_b200 import synth

pytestmark = pytest.mark.gpu

from gpu_helpers import bf16_to_f64, to_dev_bf16


@pytest.fixture(scope="module")
def native():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from nvfp4_quantized_dense_w4a16_b200 import build
    build.build()
    from nvfp4_quantized_dense_w4a16_b200 import native as N
    return N


@pytest.fixture(autouse=True)
def no_device_error(native):
    yield
    torch.cuda.synchronize()
    assert native.ffn_nvfp4_device_error(clear=False) == 0


# ------------------------------------------------------------------- routing

def check_route(native, logits, bias=None, dtype=torch.float32, **kw):
    """Ids equal the oracle's, weights within their rounding.

    Tolerance of a weight, in half steps of fp32 (2^-24 relative): exp in fp32
    of a rounded difference l - max costs |d| e^d <= 1/e of a half step of the
    sum and 4 for the function, the tree of the sum E/32 + 5 additions, the
    quotient, the scale and the last rounding 3: E/32 + 13.
    """
    l = torch.as_tensor(np.asarray(logits, dtype=np.float32)).to(dtype)
    b = None if bias is None else torch.as_tensor(np.asarray(bias, dtype=np.float32))
    ids, w = native.ffn_nvfp4_moe_route(l.cuda(), bias=None if b is None else b.cuda(), **kw)
    torch.cuda.synchronize()
    rid, rw = M.route(l.double().numpy(), None if b is None else b.double().numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = w.double().cpu().numpy()
    tol = (l.shape[1] / 32 + 13) * 2.0 ** -24
    assert np.all(np.abs(got - rw) <= tol * np.abs(rw) + 2.0 ** -149), np.max(np.abs(got - rw) / np.maximum(np.abs(rw), 1e-300))
    return ids, w


@pytest.mark.parametrize("m,experts,kw", [
    (1, 1, dict(top_k=1)),
    (1, 64, dict(top_k=8)),
    (5, 31, dict(top_k=31)),
    (37, 33, dict(top_k=5, scoring="sigmoid", renormalize=False, scale=2.5)),
    (64, 128, dict(top_k=8, renormalize=False)),
    (70, 160, dict(top_k=6, groups=8, top_groups=3, group_score="max")),
    (129, 256, dict(top_k=8, scoring="sigmoid", groups=8, top_groups=4, group_score="top2", scale=2.5)),
    (33, 96, dict(top_k=4, groups=32, top_groups=2, group_score="top2")),
    (9, 257, dict(top_k=32, scoring="sigmoid")),
    (3, 1024, dict(top_k=32)),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_matches_oracle(native, m, experts, kw, dtype, with_bias):
    rng = np.random.default_rng(1000 + m + experts)
    logits = 2.0 * rng.standard_normal((m, experts))
    bias = 0.1 * rng.standard_normal(experts) if with_bias else None
    check_route(native, logits, bias, dtype, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest_id(native, scoring):
    rng = np.random.default_rng(7)
    logits = rng.integers(-2, 3, (64, 96)).astype(np.float64)  # many equal logits
    check_route(native, logits, None, top_k=9, scoring=scoring)
    check_route(native, logits, np.zeros(96), top_k=9, scoring=scoring, groups=6, top_groups=2, group_score="top2")
    check_route(native, np.zeros((3, 64)), None, top_k=8, scoring=scoring, groups=4, top_groups=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_decides_as_64_bits(native, scoring):
    """Keys a few fp32 steps apart, or less than one: the bias cancels the score up to a remainder."""
    rng = np.random.default_rng(8)
    experts = 64
    logits = np.sort(rng.standard_normal((256, experts)).astype(np.float32), axis=1)
    score = np.exp(M.log_score(logits[0], scoring))
    bias = (1.0 - score).astype(np.float32)  # row 0: all keys within 2^-24 of one another
    logits[1:128] = logits[0]
    step = np.float32(2.0 ** -23)
    logits[1:64] *= 1 + step * rng.integers(-1, 2, (63, experts)).astype(np.float32)
    check_route(native, logits, bias, top_k=8, scoring=scoring)
    check_route(native, logits, bias, top_k=6, scoring=scoring, groups=8, top_groups=3, group_score="top2")
    check_route(native, logits, bias, top_k=6, scoring=scoring, groups=8, top_groups=3, group_score="max")
    # sigmoids that round to one in fp32
    big = rng.uniform(15.0, 22.0, (64, experts)).astype(np.float32)
    check_route(native, big, None, top_k=8, scoring=scoring)
    check_route(native, big, np.zeros(experts), top_k=8, scoring=scoring, groups=4, top_groups=2, group_score="top2")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masked_experts(native, scoring, groups):
    rng = np.random.default_rng(9)
    logits = rng.standard_normal((40, 32))
    logits[rng.random((40, 32)) < 0.85] = -np.inf
    logits[0] = -np.inf
    logits[1] = -np.inf
    logits[1, 17] = 0.5
    logits[2] = np.finfo(np.float32).min
    logits[3, :] = -np.inf
    logits[3, :8] = -200.0 - np.arange(8)  # scores that underflow keep their ratio
    kw = dict(top_k=6, scoring=scoring, groups=groups, top_groups=max(1, groups // 2), group_score="top2")
    check_route(native, logits, None, **kw)
    bias = 0.1 * rng.standard_normal(32)
    bias[5] = -np.inf
    check_route(native, logits, bias, **kw)
    check_route(native, logits, None, renormalize=False, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_group_scores_that_cancel(native, scoring):
    """Groups whose two best keys are large and of opposite sign: their sum keeps little of fp32."""
    rng = np.random.default_rng(11)
    experts, groups = 64, 8
    size = experts // groups
    logits = rng.standard_normal((200, experts)).astype(np.float32)
    bias = np.full(experts, -np.inf, np.float32)
    for g in range(groups):
        big = 0.0 if g % 2 else 3.0e5 * (g + 1)
        bias[g * size + g] = big + (0.0 if big else 0.25)
        bias[g * size + (g + 3) % size] = -big + (0.0 if big else 0.25)
    check_route(native, logits, bias, top_k=4, scoring=scoring, groups=groups, top_groups=2, group_score="top2")


def test_route_scores_below_the_normal_range(native):
    """Softmax scores around fp32's smallest numbers decide as 64-bit ones do.  A weight of theirs is off by some of
    the smallest steps (2^-149): two of the exponential, one of its product, doubled by a sum of one half, one of the
    quotient."""
    rng = np.random.default_rng(12)
    logits = rng.uniform(-104.0, -86.0, (100, 64)).astype(np.float32)
    logits[:, 10] = 0.0
    for bias, kw in ((None, dict(groups=4, top_groups=2, group_score="top2")), (np.zeros(64, np.float32), {}),
                     (None, dict(scoring="sigmoid", groups=4, top_groups=2, group_score="top2"))):
        ids, w = native.ffn_nvfp4_moe_route(torch.from_numpy(logits).cuda(), 8,
                                            bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
        rid, rw = M.route(logits.astype(np.float64), bias, 8, **kw)
        assert np.array_equal(ids.cpu().numpy(), rid)
        assert np.all(np.abs(w.double().cpu().numpy() - rw) <= 15 * 2.0 ** -24 * rw + 8 * 2.0 ** -149)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,big,top_k", [(8, 1, 1), (40, 2, 4), (64, 1, 8), (128, 3, 31), (200, 2, 8), (700, 3, 6)])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_large_errors_behind_the_choice(native, scoring, experts, big, top_k, groups):
    """A score near one that its bias cancels has an error far beyond that of the tiny keys it stands among: however far
    behind them it seems to stand, it may belong in front."""
    rng = np.random.default_rng(21 + experts)
    rows = 60
    logits = rng.uniform(-10.0, -9.9, (rows, experts)).astype(np.float32)
    where = rng.permutation(experts)[:big]
    logits[:, where] = rng.uniform(1.0, 3.0, big)
    logits[rows // 2:, :] = logits[0]  # half of them but for the cancelled experts the same
    logits[rows // 2:, where] += rng.uniform(-1e-7, 1e-7, (rows - rows // 2, big))
    score = np.exp(M.log_score(logits[0].astype(np.float64), scoring))
    bias = (1e-4 + 6e-8 * rng.uniform(-1.0, 1.0, experts) - score).astype(np.float32)
    kw = dict(top_k=top_k, scoring=scoring, groups=groups, top_groups=max(1, groups - 1), group_score="max")
    check_route(native, logits, bias, **kw)
    # equal tiny keys, so that the choice ends among equal ones
    bias[:] = 1e-4
    logits[:] = -10.0
    logits[:, where] = rng.uniform(1.0, 3.0, big)
    score = np.exp(M.log_score(logits[0].astype(np.float64), scoring))
    rest = np.setdiff1d(np.arange(experts), where)
    bias[where] = bias[rest[0]] + score[rest[0]] - score[where] + 3e-8 * rng.uniform(-1.0, 1.0, big)
    check_route(native, logits, bias, **kw)


def test_route_large_errors_by_hand(native):
    """Rows whose last key in fp32 is the first one in fact."""
    for logits, bias, best in (
            ([2.15468, -9.210265, -9.210468], [-0.8960053, 0.0, 0.0], 0),
            ([-30.0, -30.0, 6.491729259490967], [0.009999999776482582, 0.009999992325901985, -0.9884862899780273], 2)):
        ids, _ = check_route(native, [logits], bias, top_k=1, scoring="sigmoid")
        assert ids.tolist() == [[best]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_peaked_and_equal_rows(native, scoring):
    """One score near one beside many small and close ones, rows of one logit, few distinct logits."""
    rng = np.random.default_rng(22)
    logits = rng.uniform(-9.0, -8.9, (64, 160)).astype(np.float32)
    logits[:, 77] = 8.0
    logits[::2, 20:] = logits[::2, :1]
    logits[5] = 0.25
    bias = (1e-4 * rng.standard_normal(160)).astype(np.float32)
    for b in (bias, np.zeros(160, np.float32), np.full(160, 1e6, np.float32)):
        check_route(native, logits, b, top_k=8, scoring=scoring)
        check_route(native, logits, b, dtype=torch.bfloat16, top_k=13, scoring=scoring)
        check_route(native, logits, b, top_k=8, scoring=scoring, groups=8, top_groups=3, group_score="top2")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring,low,high", [("sigmoid", 30.0, 60.0), ("sigmoid", -900.0, -700.0), ("sigmoid", -1e-8, 1e-8),
                                              ("softmax", -900.0, -700.0), ("softmax", -1e-17, 1e-17)])
def test_route_scores_that_64_bits_do_not_tell_apart(native, dtype, scoring, low, high):
    """Scores that saturate, underflow or round to one number: the logits' order decides, with no bias as with one that
    is the same for all experts, in the groups' scores as well; of equal logits the lower id."""
    rng = np.random.default_rng(23)
    logits = rng.uniform(low, high, (40, 96)).astype(np.float32)
    logits[20:] = rng.choice(logits[0, :7], (20, 96))
    if scoring == "softmax":
        logits[:, 50] = 1.0
    for kw in (dict(top_k=9), dict(top_k=32), dict(top_k=6, groups=8, top_groups=3, group_score="max"),
               dict(top_k=6, groups=6, top_groups=2, group_score="max"), dict(top_k=6, groups=3, top_groups=2, group_score="max")):
        rid, _ = M.route(torch.from_numpy(logits).to(dtype).double().numpy(), None, scoring=scoring, **kw)
        for bias in (None, np.zeros(96), np.full(96, 0.25), np.full(96, -3.0)):
            b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
            ids, _ = native.ffn_nvfp4_moe_route(torch.from_numpy(logits).to(dtype).cuda(), bias=b, scoring=scoring, **kw)
            assert np.array_equal(ids.cpu().numpy(), rid), (kw, bias is None)


def test_route_equal_keys_by_hand(native):
    for scoring, logits, top_k, want in (("sigmoid", [38.0, 40.0], 1, [1]), ("sigmoid", [40.0, 50.0, 50.0], 2, [1, 2]),
                                         ("softmax", [-800.0, -790.0, 0.0], 2, [2, 1]), ("softmax", [0.0, -800.0, -790.0], 2, [0, 2])):
        for bias in (None, np.zeros(len(logits))):
            ids, _ = check_route(native, [logits], bias, top_k=top_k, scoring=scoring)
            assert ids.tolist() == [want]
    # equal infinite keys by the id
    ids, _ = check_route(native, [[1.0, 2.0, 3.0]], [np.inf, 0.0, np.inf], top_k=2, scoring="sigmoid")
    assert ids.tolist() == [[0, 2]]


@pytest.mark.parametrize("top", [-90.0, -60.5, -59.5, -40.0, -25.0])
def test_route_sigmoids_below_the_normal_range_keep_their_ratio(native, top):
    """Renormalised sigmoids of logits so low that fp32 holds their scores in few bits, or not at all, beside a better
    one: the weights are ratios and far from that."""
    rng = np.random.default_rng(24)
    logits = rng.uniform(top - 80.0, top, (50, 40))
    logits[:, 11] = top
    check_route(native, logits, None, top_k=12, scoring="sigmoid")
    check_route(native, logits, np.zeros(40), top_k=12, scoring="sigmoid", scale=2.5)
    logits[:, 30] = 4.0  # from here on to the smallest numbers
    ids, w = native.ffn_nvfp4_moe_route(torch.from_numpy(logits.astype(np.float32)).cuda(), 12, scoring="sigmoid")
    rid, rw = M.route(logits.astype(np.float32).astype(np.float64), None, 12, scoring="sigmoid")
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.all(np.abs(w.double().cpu().numpy() - rw) <= 15 * 2.0 ** -24 * rw + 4 * 2.0 ** -149)


def test_route_infinite_keys(native):
    """+inf biases tie by id; +inf logits under sigmoid score one; biases and logits of -inf close an expert."""
    rng = np.random.default_rng(13)
    logits = rng.standard_normal((20, 48)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(48)).astype(np.float32)
    bias[[30, 7, 19]] = np.inf
    bias[[3, 31]] = -np.inf
    logits[5, 7] = -np.inf
    check_route(native, logits, bias, top_k=5)
    check_route(native, logits, bias, top_k=5, groups=6, top_groups=3, group_score="top2")
    logits[2, [4, 40, 30]] = np.inf
    check_route(native, logits, bias, top_k=5, scoring="sigmoid")
    check_route(native, logits, None, top_k=5, scoring="sigmoid")
    check_route(native, np.zeros((2, 32)), np.linspace(0, 1, 32), top_k=32, scoring="sigmoid")


def test_route_non_finite_rows(native):
    logits = np.random.default_rng(10).standard_normal((6, 40)).astype(np.float32)
    logits[1, 3] = np.nan
    logits[2] = np.nan
    logits[4, 7] = np.inf
    for scoring in ("softmax", "sigmoid"):
        ids, w = native.ffn_nvfp4_moe_route(torch.from_numpy(logits).cuda(), 4, scoring=scoring)
        ids, w = ids.cpu().numpy(), w.cpu().numpy()
        bad = [1, 2, 4] if scoring == "softmax" else [1, 2]
        for i in range(6):
            assert np.all(np.isnan(w[i])) if i in bad else np.all(np.isfinite(w[i]))
        assert ids[2].tolist() == [-1] * 4 and 3 not in ids[1] and ids[4, 0] == 7
        good = [i for i in range(6) if i not in bad]
        rid, _ = M.route(logits[good].astype(np.float64), None, 4, scoring=scoring)
        assert np.array_equal(ids[good], rid)
    nan_bias = np.zeros(32, np.float32)
    nan_bias[11] = np.nan
    ids, w = native.ffn_nvfp4_moe_route(torch.from_numpy(logits[:1, :32]).cuda(), 32, bias=torch.from_numpy(nan_bias).cuda())
    assert 11 not in ids.cpu().numpy() and ids[0, 31].item() == -1 and bool(torch.isfinite(w).all())


def test_route_strided_rows_and_streams(native):
    wide = torch.randn((50, 200), generator=torch.Generator().manual_seed(3))
    part = wide.cuda()[:, 3:67]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids, w = native.ffn_nvfp4_moe_route(part, 8, stream=s)
    s.synchronize()
    rid, _ = M.route(wide[:, 3:67].double().numpy(), None, 8)
    assert np.array_equal(ids.cpu().numpy(), rid)
    empty = native.ffn_nvfp4_moe_route(part[:0], 8)
    assert empty[0].shape == (0, 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("experts,start,width", [(128, 1, 130), (256, 8, 264), (64, 2, 70), (512, 4, 520)])
def test_route_rows_off_the_wide_boundaries(native, dtype, experts, start, width):
    wide = torch.randn((33, width), generator=torch.Generator().manual_seed(experts)).to(dtype)
    part = wide.cuda()[:, start:start + experts]
    ids, w = native.ffn_nvfp4_moe_route(part, 8, groups=4, top_groups=2)
    rid, rw = M.route(wide[:, start:start + experts].double().numpy(), None, 8, groups=4, top_groups=2)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.allclose(w.double().cpu().numpy(), rw, rtol=(experts / 32 + 13) * 2.0 ** -24, atol=0)


def test_route_refusals(native):
    l = torch.zeros((4, 32), device="cuda")
    with pytest.raises(TypeError):
        native.ffn_nvfp4_moe_route(l.half(), 4)
    with pytest.raises(ValueError):
        native.ffn_nvfp4_moe_route(l.cpu(), 4)
    with pytest.raises(ValueError):
        native.ffn_nvfp4_moe_route(l.t(), 4)
    with pytest.raises(ValueError):
        native.ffn_nvfp4_moe_route(l, 4, bias=torch.zeros(31, device="cuda"))
    with pytest.raises(native.FfnError) as e:
        native.ffn_nvfp4_moe_route(l, 33)
    assert e.value.status_name == "FFN_ERR_SHAPE"


# ------------------------------------------------------------ experts' products

class Stack:
    """Random NVFP4 experts on both sides: any code, scales over several binades (some zero), tensor scales."""

    def __init__(self, native, experts, n, k, seed, gate_up=False):
        rng = np.random.default_rng(seed)
        codes = rng.integers(0, 256, (experts, n, k // 2), dtype=np.uint8)
        scales = rng.integers(0x28, 0x48, (experts, n, k // 16), dtype=np.uint8)
        scales[rng.random(scales.shape) < 0.02] = 0
        parts = 2 if gate_up else 1
        gs = (rng.uniform(0.5, 2.0, (experts, parts)) / (5.0 * np.sqrt(k))).astype(np.float32)
        self.w = M.experts_dequant(codes, scales, gs)
        dev = lambda a: torch.from_numpy(a).cuda()
        self.handle = native.ffn_nvfp4_experts_create(dev(codes), dev(scales), dev(gs if gate_up else gs[:, 0].copy()),
                                                      gate_up=gate_up)


def rows(m, k, seed):
    bits = synth.random_bf16((m, k), seed)
    return to_dev_bf16(bits), synth.bf16_bits_to_f32(bits).astype(np.float64)


def pick(rng, m, experts, top_k, padding=0.0, favourite=None):
    ids = np.stack([rng.choice(experts, top_k, replace=False) for _ in range(m)]).astype(np.int32) if m else np.zeros((0, top_k), np.int32)
    if favourite is not None:
        ids[:, 0] = favourite
    ids[rng.random(m) < padding] = -1
    return ids


def sum_error(k):
    """Relative error of a product's fp32 sum to the sum of the terms' magnitudes.

    The terms (8-bit times 6-bit significands) are exact; the tensor core adds 16 (or 64) at a time, each such step
    losing at most one step of fp32 in alignment and one in rounding (2^-22 together); the partial sums of at most 64
    ranges of K, the tensor scale and its product add 66 half steps."""
    return (k / 16 + 33) * 2.0 ** -22


HALF = 2.0 ** -8  # half a step of bf16, relative


def check_linear(native, stack, x, x64, ids, **kw):
    y = native.ffn_nvfp4_experts_linear(x, stack.handle, torch.from_numpy(ids).cuda(), **kw)
    torch.cuda.synchronize()
    ref = M.experts_linear(x64, stack.w, ids)
    tol = sum_error(x64.shape[1]) * M.experts_linear(np.abs(x64), np.abs(stack.w), ids)
    got = bf16_to_f64(y)
    err = np.abs(got - ref)
    bound = HALF * np.abs(ref) + (1 + HALF) * tol + 2.0 ** -133
    assert np.all(err <= bound), (float((err / np.maximum(bound, 1e-300)).max()), np.unravel_index(np.argmax(err - bound), err.shape))
    return y


@pytest.mark.parametrize("m,experts,top_k,n,k,padding", [
    (1, 1, 1, 8, 32, 0.0), (1, 4, 4, 128, 64, 0.0), (1, 8, 2, 200, 96, 0.0), (2, 5, 3, 129, 160, 0.0),
    (9, 3, 2, 64, 1056, 0.3), (17, 20, 3, 1000, 256, 0.1), (40, 2, 2, 384, 512, 0.0), (70, 6, 1, 33, 128, 0.2),
    (130, 3, 2, 256, 320, 0.1), (300, 2, 1, 136, 2048, 0.0), (600, 7, 4, 128, 192, 0.05),
])
def test_linear_matches_oracle(native, m, experts, top_k, n, k, padding):
    rng = np.random.default_rng(2000 + m)
    s = Stack(native, experts, n, k, 2100 + m)
    x, x64 = rows(m, k, 2200 + m)
    check_linear(native, s, x, x64, pick(rng, m, experts, top_k, padding))


@pytest.mark.parametrize("m", [1, 5, 64, 300])
def test_linear_uneven_experts(native, m):
    """All rows at one expert, none at most others; ids outside the stack; the same id twice in a row."""
    s = Stack(native, 9, 144, 224, 31)
    x, x64 = rows(m, 224, 32)
    ids = np.full((m, 3), 6, np.int32)
    check_linear(native, s, x, x64, ids)
    ids[:, 1] = 9
    ids[:, 2] = -2**31
    check_linear(native, s, x, x64, ids)
    none = torch.full((m, 3), -1, dtype=torch.int32, device="cuda")
    y = torch.full((m, 3, 144), float("nan"), dtype=torch.bfloat16, device="cuda")
    native.ffn_nvfp4_experts_linear(x, s.handle, none, y=y)
    assert int(torch.count_nonzero(y.view(torch.int16))) == 0


@pytest.mark.parametrize("m,n,k,experts,top_k,padding", [
    # a plan of few and of many pairs per expert, made by one CTA and by several
    (32, 72, 96, 3, 1, 0.0), (33, 72, 96, 3, 1, 0.0), (35, 136, 64, 7, 1, 0.0), (36, 136, 64, 7, 1, 0.1),
    (56, 136, 64, 7, 1, 0.0), (57, 136, 64, 7, 1, 0.1), (70, 136, 64, 7, 1, 0.0), (71, 136, 64, 7, 1, 0.1), (700, 64, 32, 1024, 6, 0.1), (2049, 72, 96, 17, 2, 0.1),
    (4096, 40, 32, 2, 1, 0.0), (4097, 40, 32, 2, 1, 0.3),
])
def test_linear_at_the_kernels_boundaries(native, m, n, k, experts, top_k, padding):
    rng = np.random.default_rng(2300 + m)
    s = Stack(native, experts, n, k, 2400 + m)
    x, x64 = rows(m, k, 2500 + m)
    check_linear(native, s, x, x64, pick(rng, m, experts, top_k, padding))


@pytest.mark.parametrize("k", [32, 64, 96, 128, 544])
@pytest.mark.parametrize("n", [1, 63, 130, 260])
def test_linear_many_rows_any_depth(native, n, k):
    """Row tiles of even sizes around the largest, odd numbers of K chunks, and as many tiles as keep every stage of
    the pipeline in turn; columns that no vector store fits."""
    rng = np.random.default_rng(2600 + n + k)
    s = Stack(native, 2, n, k, 2700 + n + k)
    m = 1100
    x, x64 = rows(m, k, 2800 + k)
    ids = np.zeros((m, 1), np.int32)
    ids[rng.permutation(m)[:300]] = 1
    check_linear(native, s, x, x64, ids)


@pytest.mark.parametrize("m", [3, 64])
def test_linear_every_code_and_scale(native, m):
    """Rows with a single one in them read the weight itself: every code with every scale, subnormal ones included,
    in every place of a chunk."""
    n, k = 200, 224
    rng = np.random.default_rng(43)
    codes = rng.integers(0, 256, (2, n, k // 2), dtype=np.uint8)
    scales = np.resize(np.arange(0x7F, dtype=np.uint8), 2 * n * (k // 16))
    scales = rng.permutation(scales).reshape(2, n, k // 16)
    gs = np.array([1.0, 0.5], np.float32)
    w = M.experts_dequant(codes, scales, gs)
    h = native.ffn_nvfp4_experts_create(*(torch.from_numpy(a).cuda() for a in (codes, scales, gs)))
    ids = np.tile(np.array([[1, 0]], np.int32), (m, 1))
    for k0 in range(0, k, m):
        xi = np.zeros((m, k))
        for i in range(m):
            xi[i, (k0 + i) % k] = 1.0
        y = native.ffn_nvfp4_experts_linear(torch.from_numpy(xi).to(torch.bfloat16).cuda(), h, torch.from_numpy(ids).cuda())
        assert np.array_equal(bf16_to_f64(y), M.experts_linear(xi, w, ids))


def test_linear_offsets_past_32_bits(native):
    """Weights of more than 4 GB and outputs of more than 2^31 elements: the far ends are where they belong."""
    experts, n, k = 600, 16384, 1024
    gen = torch.Generator("cuda").manual_seed(44)
    codes = torch.randint(0, 256, (experts, n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(0x30, 0x40, (experts, n, k // 16), dtype=torch.uint8, device="cuda", generator=gen)
    gs = torch.full((experts,), 2.0 ** -6, device="cuda")
    h = native.ffn_nvfp4_experts_create(codes, scales, gs)
    w = {e: M.experts_dequant(codes[e:e + 1].cpu().numpy(), scales[e:e + 1].cpu().numpy(), gs[:1].cpu().numpy())[0]
         for e in (599, 511)}
    del codes, scales
    m = 70000
    x, x64 = rows(m, k, 45)
    for count in (1, 40, m):
        ids = torch.full((count, 2), -1, dtype=torch.int32)
        ids[:, 0] = torch.arange(count) % 97
        ids[0, 1], ids[count - 1, 0] = 511, 599
        y = native.ffn_nvfp4_experts_linear(x[:count], h, ids.cuda())
        for i, j, e in ((0, 1, 511), (count - 1, 0, 599)):
            ref, mag = w[e] @ x64[i], np.abs(w[e]) @ np.abs(x64[i])
            got = bf16_to_f64(y[i, j])
            assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + (1 + HALF) * sum_error(k) * mag)
        if count > 1:
            assert int(torch.count_nonzero(y[count - 1, 1])) == 0


def test_linear_exact_integers(native):
    """Small whole numbers: every product and sum is exact, so the bits are the oracle's."""
    rng = np.random.default_rng(41)
    s = Stack(native, 4, 96, 128, 42)
    codes = rng.integers(0, 256, (4, 96, 64), dtype=np.uint8)
    scales = np.full((4, 96, 8), 0x38, np.uint8)  # 1.0
    gs = np.ones(4, np.float32)
    h = native.ffn_nvfp4_experts_create(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), torch.from_numpy(gs).cuda())
    w = M.experts_dequant(codes, scales, gs)
    for m in (1, 3, 90, 400):
        xi = rng.integers(-3, 4, (m, 128)).astype(np.float64)
        x = torch.from_numpy(xi).to(torch.bfloat16).cuda()
        ids = pick(rng, m, 4, 2)
        y = native.ffn_nvfp4_experts_linear(x, h, torch.from_numpy(ids).cuda())
        assert np.array_equal(bf16_to_f64(y), O.round_to_bf16(M.experts_linear(xi, w, ids)))


def test_linear_non_finite_rows_stay_their_own(native):
    s = Stack(native, 3, 128, 256, 51)
    for m in (2, 12, 200):
        x, x64 = rows(m, 256, 52)
        x[1, 17] = float("nan")
        ids = np.zeros((m, 2), np.int32)
        ids[:, 1] = 2
        y = native.ffn_nvfp4_experts_linear(x, s.handle, torch.from_numpy(ids).cuda())
        assert bool(torch.isnan(y[1]).all())
        assert bool(torch.isfinite(torch.cat([y[:1], y[2:]])).all())


# ------------------------------------------------------------------- the layer

class Layer:
    def __init__(self, native, experts, hidden, inter, seed):
        self.native, self.hidden, self.inter, self.experts = native, hidden, inter, experts
        self.gu = Stack(native, experts, 2 * inter, hidden, seed, gate_up=True)
        self.dn = Stack(native, experts, hidden, inter, seed + 1)

    def run(self, x, ids, weights, **kw):
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        return self.native.ffn_nvfp4_moe_forward(x, self.gu.handle, self.dn.handle, d(ids), d(weights), **kw)

    def check(self, out, x64, ids, weights):
        """Error carried through the layer: the products' sums, silu (slope at most 1.1, a few steps of fp32), the
        rounding of h, the down sums, the weighted sum (top_k + 1 half steps) and the last rounding."""
        top_k = ids.shape[1]
        ref = M.moe_forward(x64, self.gu.w, self.dn.w, ids, weights)
        g, u, h = M.moe_hidden(x64, self.gu.w, ids)
        mag = sum_error(self.hidden) * M.experts_linear(np.abs(x64), np.abs(self.gu.w), ids)
        dg, du = mag[:, :, :self.inter], mag[:, :, self.inter:]
        sg = np.abs(g / (1 + np.exp(-g)))
        # the bf16 value of h may fall to the other side of a midpoint: a whole step from the oracle's
        dh = (1.1 * dg * np.abs(u) + sg * du + 1.1 * dg * du + 16 * 2.0 ** -24 * np.abs(h)) * (1 + 2 * HALF) + 2 * HALF * np.abs(h)
        ref_h = h
        wd, aw = np.abs(self.dn.w), np.abs(np.asarray(weights, np.float64))
        bound = np.zeros_like(ref)
        mag_out = np.zeros_like(ref)
        for j in range(top_k):
            for i, e in enumerate(ids[:, j]):
                if 0 <= e < self.experts:
                    terms = wd[e] @ (np.abs(ref_h[i, j]) + dh[i, j])
                    bound[i] += aw[i, j] * (wd[e] @ dh[i, j] + sum_error(self.inter) * terms)
                    mag_out[i] += aw[i, j] * terms
        bound += (top_k + 1) * 2.0 ** -24 * mag_out
        bound = (1 + HALF) * bound + HALF * np.abs(ref) + 2.0 ** -133
        got = bf16_to_f64(out)
        err = np.abs(got - ref)
        assert np.all(err <= bound), float((err / bound).max())
        # the bound adds magnitudes; errors of either sign mostly cancel: two roundings to bf16 in the 2-norm
        n = np.linalg.norm(ref)
        assert n == 0 or np.linalg.norm(got - ref) <= 2 * HALF * n


@pytest.mark.parametrize("m,experts,top_k,hidden,inter,padding", [
    (1, 1, 1, 32, 32, 0.0), (1, 8, 2, 256, 96, 0.0), (1, 16, 8, 512, 160, 0.0), (1, 3, 3, 1056, 32, 0.0),
    (2, 4, 2, 128, 704, 0.0), (7, 20, 3, 352, 224, 0.2), (24, 16, 4, 256, 128, 0.0), (33, 2, 2, 160, 288, 0.1),
    (64, 5, 1, 384, 64, 0.3), (128, 4, 2, 256, 320, 0.0), (257, 3, 2, 192, 96, 0.1), (520, 2, 1, 128, 128, 0.0),
])
def test_layer_matches_oracle(native, m, experts, top_k, hidden, inter, padding):
    rng = np.random.default_rng(3000 + m)
    layer = Layer(native, experts, hidden, inter, 3100 + m)
    x, x64 = rows(m, hidden, 3200 + m)
    ids = pick(rng, m, experts, top_k, padding)
    weights = rng.uniform(0.0, 1.0, (m, top_k)).astype(np.float32)
    layer.check(layer.run(x, ids, weights), x64, ids, weights)


@pytest.mark.parametrize("m,experts,top_k,hidden,inter", [
    (1, 2, 1, 256, 2080, ), (3, 3, 2, 64, 4096), (16, 2, 2, 96, 1600), (33, 12, 1, 64, 2080), (32, 7, 1, 128, 64),
    (33, 7, 1, 128, 64), (35, 7, 1, 128, 64), (36, 7, 1, 128, 64), (56, 7, 1, 128, 64), (57, 7, 1, 128, 64),
    (70, 7, 1, 128, 64), (71, 7, 1, 128, 64), (255, 1, 1, 64, 64), (256, 1, 1, 128, 96), (257, 1, 1, 96, 32),
    (513, 2, 1, 160, 64), (640, 3, 2, 64, 128),
    (2100, 17, 2, 96, 32), (1, 64, 32, 96, 64), (2, 40, 33, 96, 64),
])
def test_layer_at_the_kernels_boundaries(native, m, experts, top_k, hidden, inter):
    """Long sums over few tiles (cut into ranges of K), and the numbers of pairs where other kernels take over."""
    rng = np.random.default_rng(3300 + m)
    layer = Layer(native, experts, hidden, inter, 3400 + m)
    x, x64 = rows(m, hidden, 3500 + m)
    ids = pick(rng, m, experts, top_k)
    weights = rng.uniform(0.0, 1.0, (m, top_k)).astype(np.float32)
    layer.check(layer.run(x, ids, weights), x64, ids, weights)


@pytest.mark.parametrize("m,experts,top_k,hidden,inter", [
    (1, 4, 2, 64, 96), (1, 8, 8, 96, 544), (1, 1, 1, 128, 64), (2, 4, 2, 64, 96), (4, 6, 3, 160, 256),
    (4, 3, 8, 64, 544), (5, 6, 3, 96, 96), (8, 7, 4, 128, 160), (16, 5, 2, 64, 320), (32, 9, 1, 96, 64),
])
def test_layer_of_few_pairs_keeps_16_bits_of_the_hidden_rows(native, m, experts, top_k, hidden, inter):
    """Up to 32 pairs h goes to the down products as two bf16 parts, off by 2^-16 of it (half a step of the second part,
    which is at most half a step of the first).

    Whole x and gate and up weights of small whole numbers make the products exact; silu and its product cost 16 half
    steps of fp32 as above, the down sums theirs.  The bound is far below half a step of bf16 of the terms, so that an
    oracle without the second part leaves it."""
    rng = np.random.default_rng(3800 + m + inter)
    codes = rng.integers(0, 256, (experts, 2 * inter, hidden // 2), dtype=np.uint8)
    scales = np.full((experts, 2 * inter, hidden // 16), 0x38, np.uint8)  # 1.0
    gs = np.full((experts, 2), 2.0 ** -6, np.float32)
    w_gu = M.experts_dequant(codes, scales, gs)
    gu = native.ffn_nvfp4_experts_create(*(torch.from_numpy(a).cuda() for a in (codes, scales, gs)), gate_up=True)
    dn = Stack(native, experts, hidden, inter, 3900 + m)
    x64 = rng.integers(-2, 3, (m, hidden)).astype(np.float64)
    ids = np.resize(pick(rng, m, experts, min(top_k, experts)).T, (top_k, m)).T  # (some experts twice in a row)
    weights = rng.uniform(0.25, 1.0, (m, top_k)).astype(np.float32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    out = native.ffn_nvfp4_moe_forward(dev(x64).to(torch.bfloat16), gu, dn.handle, dev(ids), dev(weights))
    g, u, rounded = M.moe_hidden(x64, w_gu, ids)
    h = g / (1.0 + np.exp(-g)) * u
    dh = (2.0 ** -16 + 16 * 2.0 ** -24) * np.abs(h)
    ref, bound, without = np.zeros((3, m, hidden))
    for i in range(m):
        for j, e in enumerate(ids[i]):
            w, a = dn.w[e], float(weights[i, j])
            ref[i] += a * (w @ h[i, j])
            without[i] += a * (w @ rounded[i, j])
            terms = np.abs(w) @ (np.abs(h[i, j]) + dh[i, j])
            bound[i] += a * (np.abs(w) @ dh[i, j] + (sum_error(inter) + (top_k + 1) * 2.0 ** -24) * terms)
    bound = (1 + HALF) * bound + HALF * np.abs(ref)
    err = np.abs(bf16_to_f64(out) - ref)
    assert np.all(err <= bound), float((err / bound).max())
    lost = np.abs(O.round_to_bf16(without) - ref)
    assert np.any(lost > bound), "the bound would not see the second part missing"


@pytest.mark.parametrize("m,experts,top_k,hidden,inter", [
    (40, 12, 1, 96, 160), (60, 9, 1, 64, 544), (100, 4, 2, 128, 96), (300, 3, 2, 64, 320),
])
def test_layer_of_many_pairs_rounds_the_hidden_rows_once(native, m, experts, top_k, hidden, inter):
    """Beyond 32 pairs h is rounded to bf16, once: where no midpoint between two bf16 numbers is within silu's error of
    it, to the oracle's number.  The products are exact, as above.  silu's exponential is off by 2 + 1.2 |g| steps of
    fp32 (CUDA's bound for the fast one), the sum, the quotient and the products by 5 more."""
    rng = np.random.default_rng(4000 + m)
    codes = rng.integers(0, 256, (experts, 2 * inter, hidden // 2), dtype=np.uint8)
    scales = np.full((experts, 2 * inter, hidden // 16), 0x38, np.uint8)  # 1.0
    gs = np.full((experts, 2), 2.0 ** -6, np.float32)
    w_gu = M.experts_dequant(codes, scales, gs)
    gu = native.ffn_nvfp4_experts_create(*(torch.from_numpy(a).cuda() for a in (codes, scales, gs)), gate_up=True)
    dn = Stack(native, experts, hidden, inter, 4100 + m)
    x64 = rng.integers(-2, 3, (m, hidden)).astype(np.float64)
    ids = pick(rng, m, experts, top_k)
    weights = rng.uniform(0.25, 1.0, (m, top_k)).astype(np.float32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    out = native.ffn_nvfp4_moe_forward(dev(x64).to(torch.bfloat16), gu, dn.handle, dev(ids), dev(weights))
    g, u, h = M.moe_hidden(x64, w_gu, ids)
    exact = g / (1.0 + np.exp(-g)) * u
    off = (7.0 + 1.2 * np.abs(g)) * 2.0 ** -23 * np.abs(exact)
    near = O.round_to_bf16(exact - off) != O.round_to_bf16(exact + off)
    assert near.mean() < 0.05
    dh = np.where(near, np.abs(O.round_to_bf16(exact + off).astype(np.float64) - O.round_to_bf16(exact - off)), 0.0)
    ref, bound = np.zeros((2, m, hidden))
    for i in range(m):
        for j, e in enumerate(ids[i]):
            w, a = dn.w[e], float(weights[i, j])
            ref[i] += a * (w @ h[i, j])
            terms = np.abs(w) @ (np.abs(h[i, j]) + dh[i, j])
            bound[i] += a * (np.abs(w) @ dh[i, j] + (sum_error(inter) + (top_k + 1) * 2.0 ** -24) * terms)
    bound = (1 + HALF) * bound + HALF * np.abs(ref)
    err = np.abs(bf16_to_f64(out) - ref)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("m", [1, 2, 4, 5, 8, 11, 60])
def test_layer_the_same_expert_again(native, m):
    """Equal ids in a row count each, with their own weights; all rows at one expert."""
    layer = Layer(native, 3, 160, 96, 66)
    x, x64 = rows(m, 160, 67)
    rng = np.random.default_rng(68)
    weights = rng.uniform(-1.0, 1.0, (m, 4)).astype(np.float32)
    for ids in (np.full((m, 4), 2, np.int32), np.tile(np.array([[1, 0, 1, 5]], np.int32), (m, 1))):
        layer.check(layer.run(x, ids, weights), x64, ids, weights)


@pytest.mark.parametrize("m", [4, 20, 100])
def test_layer_non_finite_rows_stay_their_own(native, m):
    layer = Layer(native, 3, 128, 96, 74)
    x, _ = rows(m, 128, 75)
    rng = np.random.default_rng(76)
    ids, w = pick(rng, m, 3, 2), rng.uniform(0, 1, (m, 2)).astype(np.float32)
    clean = layer.run(x, ids, w)
    x[2, 5] = float("inf")
    x[3] = float("nan")
    got = layer.run(x, ids, w)
    rest = [i for i in range(m) if i not in (2, 3)]
    assert torch.equal(got[rest], clean[rest]) and bool(torch.isnan(got[3]).all())


def test_calls_on_two_streams_at_once(native):
    """Layers and products of several sizes on two streams, each with its workspace: the bits of calls made alone."""
    layer = Layer(native, 8, 512, 256, 77)
    cases = []
    for i, m in enumerate((1, 6, 40, 300)):
        x, _ = rows(m, 512, 780 + i)
        rng = np.random.default_rng(790 + i)
        ids = torch.from_numpy(pick(rng, m, 8, 2)).cuda()
        w = torch.from_numpy(rng.uniform(0, 1, (m, 2)).astype(np.float32)).cuda()
        cases.append((x, ids, w))
    run = lambda c, **kw: native.ffn_nvfp4_moe_forward(c[0], layer.gu.handle, layer.dn.handle, c[1], c[2], **kw)
    alone = [run(c) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            for c in (cases if i == 0 else reversed(cases)):
                outs[i].append(run(c, stream=s))  # (its buffers belong to the stream)
    torch.cuda.synchronize()
    for i in range(2):
        for j, o in enumerate(outs[i]):
            assert torch.equal(o, alone[j % 4 if i == 0 else 3 - j % 4])


def test_graphs_that_share_a_workspace(native):
    """Two captured layers of different sizes over one workspace, replayed in turn, and an uncaptured call between."""
    layer = Layer(native, 8, 256, 160, 84)
    size = native.ffn_nvfp4_moe_workspace_size(600, 8, 8, 256, 160)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    parts = []
    for m, top_k in ((3, 2), (600, 8), (30, 2)):
        x, _ = rows(m, 256, 85 + m)
        rng = np.random.default_rng(86 + m)
        ids = torch.from_numpy(pick(rng, m, 8, top_k)).cuda()
        w = torch.from_numpy(rng.uniform(0, 1, (m, top_k)).astype(np.float32)).cuda()
        out = torch.empty((m, 256), dtype=torch.bfloat16, device="cuda")
        run = lambda x=x, ids=ids, w=w, out=out: native.ffn_nvfp4_moe_forward(
            x, layer.gu.handle, layer.dn.handle, ids, w, out=out, workspace=ws)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            want = run().clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                run()
        parts.append((graph, run, out, want))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for a in parts:
            for b in parts:
                for p in (a, b):
                    p[2].fill_(float("nan"))
                a[0].replay()
                b[1]()
                b[0].replay()
                s.synchronize()
                assert torch.equal(a[2], a[3]) and torch.equal(b[2], b[3])


@pytest.mark.parametrize("most,experts,top_k,hidden,inter", [(33, 8, 2, 256, 4096), (20, 4, 2, 256, 2048), (70, 7, 1, 128, 2080)])
def test_one_workspace_for_every_smaller_batch(native, most, experts, top_k, hidden, inter):
    """A buffer of the largest batch's size, as a server keeps it, at every batch up to that one."""
    layer = Layer(native, experts, hidden, inter, 1001)
    x, _ = rows(most, hidden, 1002)
    rng = np.random.default_rng(1003)
    ids = torch.from_numpy(pick(rng, most, experts, top_k)).cuda()
    w = torch.from_numpy(rng.uniform(0, 1, (most, top_k)).astype(np.float32)).cuda()
    size = native.ffn_nvfp4_moe_workspace_size(most, top_k, experts, hidden, inter)
    ws = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    y = torch.empty((most, top_k, hidden), dtype=torch.bfloat16, device="cuda")
    linear = native.ffn_nvfp4_experts_workspace_size(most, top_k, experts, hidden, hidden)
    plain = Stack(native, experts, hidden, hidden, 1004)
    for m in range(1, most + 1):
        args = (x[:m], layer.gu.handle, layer.dn.handle, ids[:m], w[:m])
        out = native.ffn_nvfp4_moe_forward(*args, workspace=ws[:size])
        assert torch.equal(out, native.ffn_nvfp4_moe_forward(*args))
        native.ffn_nvfp4_experts_linear(x[:m], plain.handle, ids[:m], y=y[:m], workspace=ws[:linear])
        assert torch.equal(y[:m], native.ffn_nvfp4_experts_linear(x[:m], plain.handle, ids[:m]))
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0xA5).all())


@pytest.mark.parametrize("m", [1, 20, 150])
def test_layer_padding_rows_and_canaries(native, m):
    """Rows without an expert are zeros; nothing behind row m is written; the workspace's size is enough."""
    layer = Layer(native, 4, 128, 96, 61)
    x, x64 = rows(m, 128, 62)
    ids = np.full((m, 2), -1, np.int32)
    w = np.zeros((m, 2), np.float32)
    out = torch.full((m + 3, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    size = native.ffn_nvfp4_moe_workspace_size(m, 2, 4, 128, 96)
    ws = torch.full((size + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    layer.run(x, ids, w, out=out[:m], workspace=ws[:size])
    assert int(torch.count_nonzero(out[:m].view(torch.int16))) == 0
    ids[m // 2] = (3, 1)
    w[m // 2] = (0.25, 0.75)
    layer.run(x, ids, w, out=out[:m], workspace=ws[:size])
    torch.cuda.synchronize()
    assert bool((out[m:] == 7.0).all()) and bool((ws[size:] == 0xA5).all())
    layer.check(out[:m], x64, ids, w)
    other = [i for i in range(m) if i != m // 2]
    assert int(torch.count_nonzero(out[other].view(torch.int16))) == 0


def test_layer_weight_signs_nan_and_zero(native):
    layer = Layer(native, 4, 128, 96, 63)
    x, x64 = rows(6, 128, 64)
    ids = pick(np.random.default_rng(65), 6, 4, 2)
    w = np.array([[1, -1], [0, 2], [-3, 0], [0, 0], [1, 1], [2, 2]], np.float32)
    layer.check(layer.run(x, ids, w), x64, ids, w)
    w[4, 0] = np.nan
    ids[5] = -1
    w[5, 1] = np.nan  # a NaN weight of an id that picks nothing still shows
    out = layer.run(x, ids, w)
    assert bool(torch.isnan(out[4:]).all()) and bool(torch.isfinite(out[:4]).all())


@pytest.mark.parametrize("m", [1, 40, 300])
def test_layer_repeats_its_bits_and_rows_are_independent(native, m):
    layer = Layer(native, 6, 256, 160, 71)
    x, _ = rows(m, 256, 72)
    rng = np.random.default_rng(73)
    ids, w = pick(rng, m, 6, 3), rng.uniform(0, 1, (m, 3)).astype(np.float32)
    a = layer.run(x, ids, w)
    assert torch.equal(a, layer.run(x, ids, w))
    order = rng.permutation(m)
    b = layer.run(x[torch.from_numpy(order).cuda()].contiguous(), ids[order], w[order])
    assert torch.equal(b, a[torch.from_numpy(order).cuda()])


@pytest.mark.parametrize("m", [1, 24, 200])
def test_route_then_layer_in_a_graph_on_its_own_stream(native, m):
    """The three operators as a serving step uses them: routed, computed and replayed with new rows."""
    layer = Layer(native, 8, 256, 128, 81)
    proj = Stack(native, 8, 64, 256, 83)
    s = torch.cuda.Stream()
    x = torch.empty((m, 256), dtype=torch.bfloat16, device="cuda")
    logits = torch.empty((m, 8), device="cuda")
    bias = torch.linspace(-0.1, 0.1, 8, device="cuda")
    ids = torch.empty((m, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((m, 2), device="cuda")
    out = torch.empty((m, 256), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((m, 2, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(native.ffn_nvfp4_moe_workspace_size(m, 2, 8, 256, 128), dtype=torch.uint8, device="cuda")

    def step():
        native.ffn_nvfp4_moe_route(logits, 2, scoring="sigmoid", bias=bias, groups=4, top_groups=2, group_score="top2",
                                   ids=ids, weights=w)
        native.ffn_nvfp4_moe_forward(x, layer.gu.handle, layer.dn.handle, ids, w, out=out, workspace=ws)
        native.ffn_nvfp4_experts_linear(x, proj.handle, ids, y=y, workspace=ws)

    x.zero_()
    logits.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for seed in (1, 2):
        xd, x64 = rows(m, 256, 90 + seed)
        l = np.random.default_rng(seed).standard_normal((m, 8)).astype(np.float32)
        x.copy_(xd)
        logits.copy_(torch.from_numpy(l))
        for t in (out, y, w):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        rid, rw = M.route(l.astype(np.float64), bias.double().cpu().numpy(), 2, scoring="sigmoid", groups=4, top_groups=2,
                          group_score="top2")
        assert np.array_equal(ids.cpu().numpy(), rid) and np.allclose(w.cpu().numpy(), rw, rtol=14 * 2.0 ** -24)
        layer.check(out, x64, rid, w.cpu().numpy())
        ref = M.experts_linear(x64, proj.w, rid)
        tol = HALF * np.abs(ref) + 1.01 * sum_error(256) * M.experts_linear(np.abs(x64), np.abs(proj.w), rid)
        assert np.all(np.abs(bf16_to_f64(y) - ref) <= tol)


def test_layer_refusals(native):
    layer = Layer(native, 4, 128, 96, 91)
    x, _ = rows(3, 128, 92)
    ids = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    w = torch.ones((3, 2), device="cuda")
    run = lambda gu, dn, **kw: native.ffn_nvfp4_moe_forward(x, gu, dn, ids, w, **kw)

    def status(f):
        with pytest.raises(native.FfnError) as e:
            f()
        return e.value.status_name

    other = Stack(native, 5, 128, 96, 93).handle
    assert status(lambda: run(layer.dn.handle, layer.gu.handle)) in ("FFN_ERR_INVALID_ARG", "FFN_ERR_SHAPE")
    assert status(lambda: run(layer.gu.handle, other)) == "FFN_ERR_SHAPE"
    assert status(lambda: run(layer.gu.handle, layer.dn.handle, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))) == "FFN_ERR_WORKSPACE"
    assert status(lambda: native.ffn_nvfp4_experts_linear(x, layer.gu.handle, ids)) == "FFN_ERR_UNSUPPORTED"
    with pytest.raises(TypeError):
        native.ffn_nvfp4_moe_forward(x.float(), layer.gu.handle, layer.dn.handle, ids, w)
    with pytest.raises(TypeError):
        native.ffn_nvfp4_moe_forward(x, layer.gu.handle, layer.dn.handle, ids.long(), w)
    with pytest.raises(ValueError):
        native.ffn_nvfp4_moe_forward(x, layer.gu.handle, layer.dn.handle, ids[:2], w)
    with pytest.raises(ValueError):
        native.ffn_nvfp4_experts_linear(x[:, :64].contiguous(), layer.dn.handle, ids)
    with pytest.raises(ValueError):
        native.ffn_nvfp4_experts_create(torch.zeros((2, 64, 32), dtype=torch.uint8, device="cuda"),
                                        torch.zeros((2, 64, 4), dtype=torch.uint8, device="cuda"), torch.ones(3, device="cuda"))
    empty = native.ffn_nvfp4_moe_forward(x[:0], layer.gu.handle, layer.dn.handle, ids[:0], w[:0])
    assert empty.shape == (0, 128)
