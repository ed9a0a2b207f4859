"""Order of steps in the kernels that a run on a healthy GPU cannot show: what
happens when a bounded wait expires, and where warps have to be whole."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_quantized_dense_w4a16_b200", "csrc")


def code(name):
    """The source without comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def body(text, start):
    """A function's body: from `start` to the brace that closes its first one."""
    at = text.index(start)
    depth = 0
    for i in range(text.index("{", text.index(")", at)), len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(start)


def test_the_streaming_norm_stores_nothing_of_a_copy_that_has_not_landed():
    """The group's vote on the wait stands before the first use of the row, with a way out, in the loop over the rows."""
    loop = body(code("block_norm.cu"), "block_norm_stream_kernel(const")
    loop = loop[loop.index("r += step) {"):]
    wait, use, store = loop.index("mbar_wait("), loop.index("from = ring"), loop.index("residual_out)")
    vote = loop.index("row.all(")
    assert abs(vote - wait) < 20 and wait < use < store
    assert "return;" in loop[wait:use] and "landed(s, parity)" in loop[wait:use]


def test_warps_are_whole_at_aligned_barriers():
    """bar and barrier.cluster .aligned want all lanes of a warp: behind code of single lanes stands __syncwarp()."""
    group = code("block_norm.cu")
    group = group[group.index("struct Group"):group.index("norm_factors2")]
    for barrier in ("named_bar_sync(id, threads)", "bar.red.and.pred"):
        assert all("__syncwarp();" in group[max(0, m.start() - 160):m.start()] for m in re.finditer(re.escape(barrier), group))
    tc = code("int8_tc.cu")
    kernels = tc[tc.index("int8_pair_kernel("):tc.index("PFN_cuTensorMapEncodeTiled_v12000 encode_fn")]
    for m in re.finditer(r"cluster_sync\(\);|named_bar_sync\(", kernels):
        before = kernels[:m.start()].rstrip().splitlines()[-1].strip()
        assert before.startswith(("__syncwarp();", "__syncthreads();", "tc_fence")), before


def test_rows_that_the_kernel_ahead_writes_are_not_read_only_data():
    """const __restrict__ lets a load pass the wait for the kernel ahead, and its caches keep what that kernel changes."""
    for name in ("int8_quantize.cu", "int8_gemv.cu", "int8_tc.cu", "block_norm.cu"):
        assert "__restrict__" not in code(name), name
