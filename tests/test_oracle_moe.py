"""Pins of the mixture-of-experts oracle: hand-worked routes and the identities
that tie its layer to the dense one."""
import numpy as np
import pytest

from oracle import moe as M
from oracle import nvfp4_ffn as O


def test_route_by_hand():
    l = np.log([[1.0, 4.0, 2.0, 1.0]])  # softmax = 1/8, 4/8, 2/8, 1/8
    ids, w = M.route(l, None, 2, renormalize=False, scale=2.0)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[1.0, 0.5]], rtol=1e-15)
    ids, w = M.route(l, None, 3)  # experts 0 and 3 are equal: the lower id
    assert ids.tolist() == [[1, 2, 0]] and np.allclose(w, [[4 / 7, 2 / 7, 1 / 7]], rtol=1e-15)
    # the bias decides the choice, not the weight
    ids, w = M.route(l, [1.0, 0.0, 0.0, 0.0], 2)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[0.2, 0.8]], rtol=1e-15)


def test_route_sigmoid_and_groups_by_hand():
    l = [[0.0, 3.0, 2.0, 1.0, -1.0, 2.5]]
    s = 1 / (1 + np.exp(-np.asarray(l[0])))
    ids, w = M.route(l, None, 2, scoring="sigmoid", groups=3, top_groups=1, group_score="max")
    assert ids.tolist() == [[1, 0]] and np.allclose(w[0], s[[1, 0]] / s[[1, 0]].sum(), rtol=1e-14)
    # the two best of each group: 0.5 + .95, .88 + .73, .27 + .92
    ids, _ = M.route(l, None, 2, scoring="sigmoid", groups=3, top_groups=1, group_score="top2")
    assert ids.tolist() == [[2, 3]]
    # a group with one expert left counts that one alone
    ids, _ = M.route([[-np.inf, 3.0, 2.0, -5.0]], None, 1, scoring="sigmoid", groups=2, top_groups=1, group_score="top2")
    assert ids.tolist() == [[1]]


def test_route_masked_rows():
    ids, w = M.route([[-np.inf, 1.0, -np.inf], [-np.inf] * 3], None, 2)
    assert ids.tolist() == [[1, -1], [-1, -1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]]
    ids, w = M.route([[-3e38] * 3], None, 2, scoring="sigmoid")  # scores below any number, equal ones
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.5, 0.5]]


def _experts(rng, e, n, k):
    codes = rng.integers(0, 256, (e, n, k // 2), dtype=np.uint8)
    scales = rng.integers(0x30, 0x40, (e, n, k // 16), dtype=np.uint8)
    return codes, scales


def test_linear_is_the_dense_projection():
    rng = np.random.default_rng(5)
    codes, scales = _experts(rng, 3, 8, 32)
    gs = np.array([0.5, 2.0, 1.0])
    x = rng.integers(-4, 5, (4, 32)).astype(np.float64)
    ids = np.array([[2, 0], [1, 1], [-1, 2], [0, 3]])
    y = M.experts_linear(x, M.experts_dequant(codes, scales, gs), ids)
    for i in range(4):
        for j in range(2):
            e = ids[i, j]
            want = O.project_w4a16(x[i:i + 1], codes[e], scales[e], gs[e])[0] if 0 <= e < 3 else np.zeros(8)
            assert np.array_equal(y[i, j], want)


def test_layer_of_one_expert_is_the_dense_layer():
    rng = np.random.default_rng(6)
    h, inter = 64, 32
    gu, dn = _experts(rng, 1, 2 * inter, h), _experts(rng, 1, h, inter)
    x = O.round_to_bf16(rng.standard_normal((3, h)))
    wgu, wd = M.experts_dequant(*gu, [[0.004, 0.002]]), M.experts_dequant(*dn, [0.01])
    out = M.moe_forward(x, wgu, wd, np.zeros((3, 1), np.int32), np.ones((3, 1)))
    g, u = x @ wgu[0, :inter].T, x @ wgu[0, inter:].T
    want = O.round_to_bf16(g / (1 + np.exp(-g)) * u) @ wd[0].T
    assert np.allclose(out, want, rtol=1e-12, atol=1e-14)
    # two picks of the same expert add their weights
    two = M.moe_forward(x, wgu, wd, np.zeros((3, 2), np.int32), np.full((3, 2), 0.5))
    assert np.allclose(two, out, rtol=1e-12)


def test_route_orders_equal_scores_by_their_logits():
    """Scores that 64 bits do not tell apart, with no bias and with one for all; infinite keys by the id."""
    for bias in (None, np.zeros(3), np.full(3, 0.5)):
        assert M.route([[38.0, 40.0, 40.0]], bias, 2, scoring="sigmoid")[0].tolist() == [[1, 2]]
        assert M.route([[-800.0, -790.0, 0.0]], bias, 2)[0].tolist() == [[2, 1]]
    for bias in (None, np.zeros(4)):
        ids, _ = M.route([[40.0, 30.0, 50.0, 41.0]], bias, 2, scoring="sigmoid", groups=2, top_groups=1, group_score="max")
        assert ids.tolist() == [[2, 3]]
    assert M.route([[1.0, 2.0, 3.0]], [np.inf, 0.0, np.inf], 2, scoring="sigmoid")[0].tolist() == [[0, 2]]
