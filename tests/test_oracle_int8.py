"""The oracle of the 8-bit integer layers and the norms, on hand-worked numbers."""
import numpy as np

from oracle import int8 as I


def test_quantize_by_hand():
    # a = 127: the codes are the values rounded to even; a = 254: halves, ties to even
    codes, scales = I.quantize_rows([[127, -127, 0.5, 1.5, -2.5, 63.25], [254, 1, 3, 5, -7, -254], [0] * 6])
    assert codes.tolist() == [[127, -127, 0, 2, -2, 63], [127, 0, 2, 2, -4, -127], [0] * 6]
    assert scales.tolist() == [1.0, 2.0, 0.0]


def test_quantize_at_the_ends_of_the_range():
    tiny, big = 2.0 ** -133, float(np.float32(3.3895314e38))  # the smallest and the largest bf16 number
    codes, scales = I.quantize_rows([[tiny, -tiny, 0], [big, -big / 2, 0], [np.inf, 1, 2], [1, np.nan, 2]])
    assert codes.tolist() == [[127, -127, 0], [127, -64, 0], [0] * 3, [0] * 3]
    assert scales[0] > 0 and np.isfinite(scales[1]) and np.isnan(scales[2]) and np.isnan(scales[3])


def test_linear_by_hand():
    xq, wq = np.array([[1, -2, 3]], np.int8), np.array([[4, 5, 6], [-128, 127, 0]], np.int8)
    y = I.linear(xq, np.array([0.5], np.float32), wq, np.array([2.0, 0.25], np.float32), np.array([1.0, -1.0]))
    assert y.tolist() == [[12 * 0.5 * 2 + 1, -382 * 0.5 * 0.25 - 1]]


def test_the_largest_sum_fits_32_bits():
    assert 128 * 128 * 131040 < 2 ** 31


def test_norms_by_hand():
    v = [[3.0, -4.0]]
    assert np.allclose(I.norm(v, eps=0.0), [[3 / np.sqrt(12.5), -4 / np.sqrt(12.5)]], rtol=1e-15)
    assert np.allclose(I.norm(v, [1.0, 2.0], [0.5, 0.0], kind="layer", eps=0.0, offset=1.0), [[2.5, -3.0]], rtol=1e-15)
    assert np.allclose(I.residual([[2.0]], [[4.0]], [[0.0]], "sigmoid", 0.5, 2.0), [[5.0]], rtol=1e-15)
