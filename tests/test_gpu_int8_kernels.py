"""The kernels that 8-bit integer layers of real sizes take, on the GPU: clusters
that cut K (decode batches), wide tiles and pairs of CTAs that take several
(prompts), several blocks of weight rows of one token."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_int8 import check_forward, check_linear, layer, native, no_device_error, rows, same_bits  # noqa: F401


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


def test_decode_batches_take_clusters(native):
    """What the two tests above are for, on this GPU."""
    for m, hidden, inter in CLUSTERS:
        assert native.ffn_int8_projection_plan(m, 2 * inter, hidden, "gate_up")["kernel"] == "clusters", (m, hidden, inter)
    for hidden, inter in ((4096, 96), (8192, 160), (2048, 9632)):
        kernels = [native.ffn_int8_projection_plan(m, 2 * inter, hidden, "gate_up")["kernel"] for m in (1, 16, 48, 600)]
        assert kernels == ["row", "clusters", "clusters", "pairs"]


#: Plain products by pairs of CTAs: (m, n, k), the tile's columns, the tiles that a pair takes at most.  Columns that end
#: inside a tile, odd widths; rings that wrap inside a tile and over its end.
PAIRS = [(260, 201, 64, 64, 1), (260, 2409, 64, 96, 1), (260, 3561, 64, 128, 1), (260, 4809, 64, 160, 1), (260, 11913, 64, 192, 2),
         (260, 7113, 160, 224, 1), (260, 8361, 160, 256, 1), (513, 9417, 64, 128, 3), (513, 11049, 64, 160, 3), (513, 12585, 64, 192, 3),
         (1100, 8457, 64, 224, 3), (1100, 9897, 64, 256, 3), (1100, 9896, 1056, 256, 3), (1500, 9000, 128, 256, 3)]


@pytest.mark.parametrize("m,n,k,columns,turns", PAIRS)
def test_products_by_pairs(native, m, n, k, columns, turns):
    p = native.ffn_int8_projection_plan(m, n, k)
    assert p["kernel"] == "pairs" and p["tile_columns"] == columns and p["turns"] >= turns
    check_linear(native, m, n, k, with_bias=n % 2 == 0, seed=n)


#: Gate and up products by pairs: (m, hidden, inter), the tile's weight rows, the tiles that a pair takes.
GATE_UP_PAIRS = [(260, 64, 192, 64, 1), (260, 64, 1248, 96, 1), (260, 64, 1824, 128, 1), (260, 64, 2400, 160, 1), (1100, 64, 3744, 128, 4),
                 (260, 64, 8352, 160, 3), (260, 64, 9504, 192, 3), (260, 64, 10752, 224, 3), (260, 64, 12480, 256, 3), (700, 672, 8704, 256, 3)]


@pytest.mark.parametrize("m,hidden,inter,columns,turns", GATE_UP_PAIRS)
def test_layers_by_pairs(native, m, hidden, inter, columns, turns):
    p = native.ffn_int8_projection_plan(m, 2 * inter, hidden, "gate_up")
    assert p["kernel"] == "pairs" and p["tile_columns"] == columns and p["turns"] >= turns
    x, weights = rows(m, hidden, m), layer(hidden, inter, 7)
    out, _ = check_forward(native, x, weights)
    one = native.ffn_int8_forward(x[m - 1:].cuda(), *(t.cuda() for t in weights))
    assert same_bits(out[m - 1:], one)


@pytest.mark.parametrize("n,k,turns", [(38000, 96, 2), (37889, 64, 2), (129001, 32, 4), (40000, 8224, 2)])
def test_products_of_one_row_in_several_blocks(native, n, k, turns):
    assert native.ffn_int8_projection_plan(1, n, k)["turns"] >= turns
    check_linear(native, 1, n, k, with_bias=True, seed=n)


@pytest.mark.parametrize("hidden,inter,turns", [(96, 19008, 2), (64, 28672, 2), (32, 60000, 4)])
def test_layers_of_one_row_in_several_blocks(native, hidden, inter, turns):
    assert native.ffn_int8_projection_plan(1, 2 * inter, hidden, "gate_up")["turns"] >= turns
    check_forward(native, rows(1, hidden, 8), layer(hidden, inter, 9))
