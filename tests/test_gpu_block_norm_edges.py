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


#: Rows of every kernel: a warp's, a CTA's, one by one, few and many, and the streaming kernel's.
PLACES = [(3, 96), (4, 1024), (5, 2048), (4, 20000), (5, 99), (3, 9001), (1500, 1037), (2100, 384), (700, 2048), (450, 5120)]


@pytest.mark.parametrize("m,hidden", [(3, 256), (4, 1024), (5, 2048), (3, 16384), (700, 2048), (450, 4096)])
def test_a_row_of_one_huge_power_of_two(native, m, hidden):
    """Its sum passes fp32's range, its scaled sums are exact: a layer norm without variance is its bias."""
    n, p = make_norm(native, hidden, "layer", torch.float32, seed=3)
    r = rows(m, hidden, 4).float()
    good = native.ffn_block_norm(r.cuda(), pre=n)[1]
    r[1] = 2.0 ** 120
    x = native.ffn_block_norm(r.cuda(), pre=n)[1]
    assert same_bits(x[1].cpu(), torch.from_numpy(p["bias"]).to(torch.bfloat16))
    assert same_bits(x[2:], good[2:]) and same_bits(x[0], good[0])
    odd = torch.empty((m, hidden + 1))  # (rows that are not whole 16 bytes)
    odd[:, 1:] = r
    x = native.ffn_block_norm(odd.cuda()[:, 1:], pre=n)[1]
    assert same_bits(x[1].cpu(), torch.from_numpy(p["bias"]).to(torch.bfloat16)) and torch.all(torch.isfinite(x))
