"""Norms around a layer on the GPU where they can go wrong: weights that are
swapped, rows of one value, infinities, calls from several threads."""
import numpy as np
import pytest
import torch

from oracle import int8 as I

pytestmark = pytest.mark.gpu

from gpu_helpers import bf16_to_f64
from test_gpu_block_norm import HALF, half_step, make_norm, norm_error
from test_gpu_int8 import native, no_device_error, rows, same_bits  # noqa: F401


@pytest.mark.parametrize("m,hidden", [(3, 96), (5, 99), (2100, 384)])
def test_a_norm_follows_its_weights(native, m, hidden):
    r = rows(m, hidden, 1).cuda()
    w, other = (torch.nn.Parameter(rows(1, hidden, s)[0].cuda()) for s in (2, 3))
    n = native.Norm(w)
    call = lambda norm: native.ffn_block_norm(r, pre=norm)[1]  # noqa: E731
    first = call(n)
    assert same_bits(first, call(native.Norm(w)))
    w.data = other.data.float()
    assert same_bits(call(n), call(native.Norm(other.data.float()))) and not same_bits(call(n), first)
    n.weight, n.eps = other, 0.5
    assert same_bits(call(n), call(native.Norm(other, eps=0.5)))
    w.data = rows(1, hidden, 4)[0]
    n = native.Norm(other)
    other.data = rows(1, hidden, 4)[0]
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(n)
