"""The kernels that 8-bit integer layers of real sizes take, on the GPU: clusters
that cut K (decode batches), wide tiles and pairs of CTAs that take several
(prompts), several blocks of weight rows of one token."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_int8 import check_forward, layer, native, no_device_error, rows, same_bits  # noqa: F401


# Layers whose gate and up products go through clusters of CTAs: cut into 8, 6 and 5 ranges of K and not at all, in one
# to four blocks of rows, columns that end inside a tile of 64 and that fill it.
CLUSTERS = [(2, 4096, 96), (48, 4096, 96), (16, 2048, 992), (100, 8192, 160), (128, 8192, 160), (200, 8192, 160), (300, 8192, 160), (511, 8192, 160),
            (7, 5120, 1536), (2, 2048, 9632)]


@pytest.mark.parametrize("m,hidden,inter", CLUSTERS)
def test_layers_of_decode_batches(native, m, hidden, inter):
    check_forward(native, rows(m, hidden, m), layer(hidden, inter, 3))


@pytest.mark.parametrize("hidden,inter", [(4096, 96), (8192, 160), (2048, 9632)])
def test_rows_of_decode_batches_do_not_depend_on_the_batch(native, hidden, inter):
    """One row on the CUDA cores, clusters of every number of blocks, pairs of CTAs: the same bits."""
    x, weights = rows(600, hidden, 5).cuda(), [t.cuda() for t in layer(hidden, inter, 6)]
    whole = native.ffn_int8_forward(x, *weights)
    for m in (1, 2, 15, 16, 17, 48, 100, 128, 129, 200, 300, 400, 512):
        assert same_bits(native.ffn_int8_forward(x[:m].contiguous(), *weights), whole[:m]), m
    for i in (1, 300, 599):
        assert same_bits(native.ffn_int8_forward(x[i:i + 1].contiguous(), *weights), whole[i:i + 1]), i
