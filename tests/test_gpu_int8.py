"""8-bit integer layers on the GPU: quantisation and projections bit for bit
against the definitions, the layer but for hidden values next to a rounding."""
import numpy as np
import pytest
import torch

from oracle import int8 as I
from oracle import nvfp4_ffn as O
from nvfp4_quantized_dense_w4a16_b200 import synth

pytestmark = pytest.mark.gpu

from gpu_helpers import bf16_to_f64, bf16_ulp, to_dev_bf16


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


def same_bits(a, b):
    a, b = a.contiguous(), b.contiguous()
    return torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32 if a.element_size() == 4 else torch.int8),
                       b.view(torch.int16 if b.element_size() == 2 else torch.int32 if b.element_size() == 4 else torch.int8))


def rows(m, k, seed):
    """bf16 rows of differing size with a few large channels."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)) * np.exp(0.5 * rng.standard_normal((m, 1))) * np.where(rng.random(k) < 0.02, 10.0, 1.0)
    return torch.from_numpy(x).to(torch.bfloat16)


def codes(n, k, seed, full=False):
    rng = np.random.default_rng(seed)
    if full:
        return torch.from_numpy(rng.integers(-128, 128, (n, k)).astype(np.int8))
    return torch.from_numpy(np.clip(np.rint(36 * rng.standard_normal((n, k))), -127, 127).astype(np.int8))


def scales(n, k, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((np.exp(0.3 * rng.standard_normal(n)) / (36 * np.sqrt(k))).astype(np.float32))


# -------------------------------------------------------------- quantisation

def check_quantize(native, x, **kw):
    c, s = native.ffn_int8_quantize(x.cuda() if not x.is_cuda else x, **kw)
    torch.cuda.synchronize()
    rc, rs = I.quantize_rows(x.float().cpu().numpy())
    assert np.array_equal(c.cpu().numpy(), rc)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    return c, s


@pytest.mark.parametrize("m,k", [(1, 32), (3, 96), (37, 1056), (5, 17408), (2, 131040), (300, 64), (1, 4096), (7, 8224), (9, 40000)])
def test_quantize(native, m, k):
    check_quantize(native, rows(m, k, m + k))


def test_quantize_extremes(native):
    tiny, big = 2.0 ** -133, 3.3895314e38
    x = torch.zeros((12, 64), dtype=torch.float64)
    x[1, 3], x[2, 5], x[3] = tiny, -big, torch.linspace(-127, 127, 64, dtype=torch.float64)
    x[4], x[5, 63], x[6, 0], x[7, 7] = big, float("nan"), float("inf"), -float("inf")
    x[8] = torch.arange(64) * 0.5  # ties
    x[8, 63] = 127
    x[9], x[10], x[11] = tiny * torch.arange(64), 2.0 ** -100 * torch.randn(64), 2.0 ** -101 * torch.randn(64)
    check_quantize(native, x.to(torch.bfloat16))


def test_quantize_of_all_bf16_values(native):
    """Every finite bf16 number, in rows of 32 of neighbouring sizes."""
    bits = np.arange(0x7f80, dtype=np.uint16)
    both = np.stack([bits, bits | 0x8000]).reshape(2, -1, 32).transpose(1, 0, 2).reshape(-1, 32)
    check_quantize(native, torch.from_numpy(both.astype(np.int16)).view(torch.bfloat16))


def test_quantize_strided_rows_and_what_is_behind_them(native):
    wide = rows(11, 512, 3).cuda()
    c = torch.full((14, 256), 55, dtype=torch.int8, device="cuda")
    s = torch.full((14,), 5.0, device="cuda")
    check_quantize(native, wide[:, 128:384], codes=c[:11], scales=s[:11])
    assert torch.all(c[11:] == 55) and torch.all(s[11:] == 5)
    check_quantize(native, wide[::2, 256:])
    check_quantize(native, rows(1, 72, 4).cuda()[:, 8:])


# ---------------------------------------------------------------- projections

def ref_linear(xq, xs, wq, ws, bias=None):
    v = I.linear(xq.numpy(), xs.numpy(), wq.numpy(), ws.numpy(), None if bias is None else bias.float().numpy())
    return torch.from_numpy(v).to(torch.bfloat16)


def check_linear(native, m, n, k, with_bias=False, full=False, seed=0):
    xq, wq, ws = codes(m, k, seed + 1, full), codes(n, k, seed + 2, full), scales(n, k, seed + 3)
    xs = scales(m, 1, seed + 4)
    bias = torch.randn(n, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16) if with_bias else None
    y = native.ffn_int8_linear(xq.cuda(), wq.cuda(), ws.cuda(), x_scales=xs.cuda(), bias=None if bias is None else bias.cuda())
    torch.cuda.synchronize()
    assert same_bits(y.cpu(), ref_linear(xq, xs, wq, ws, bias))
    return y


SIZES = [(1, 1, 32), (1, 64, 64), (1, 1000, 1056), (2, 33, 4096), (3, 129, 2048), (4, 512, 8192), (5, 17, 96), (8, 1024, 1024),
         (9, 127, 1056), (16, 128, 128), (17, 300, 640), (31, 1000, 1056), (32, 96, 160), (33, 1024, 512), (64, 257, 1024),
         (65, 130, 224), (100, 640, 2080), (128, 128, 4096), (129, 384, 288), (200, 1001, 1056), (255, 250, 64), (256, 512, 512),
         (257, 255, 96), (300, 2000, 672), (511, 640, 320), (513, 1536, 1024), (1000, 264, 416), (1030, 2056, 352)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("with_bias", [False, True])
def test_linear_matches_bit_for_bit(native, m, n, k, with_bias):
    check_linear(native, m, n, k, with_bias, seed=m + n + k)


@pytest.mark.parametrize("m,n,k", [(1, 40, 131040), (3, 24, 131040), (20, 40, 131040), (150, 24, 65536), (300, 136, 131040), (2, 30000, 64),
                                   (40, 20001, 64), (5000, 8, 64), (3000, 33, 96), (7, 8, 17408), (200, 40, 17408), (385, 72, 8192), (512, 130, 12288),
                                   (260, 129, 20000 // 32 * 32), (130, 9, 40000), (1, 3, 32768), (1, 5, 32800), (1, 7000, 8224), (1, 20001, 96)])
def test_linear_long_axes(native, m, n, k):
    check_linear(native, m, n, k, full=True, seed=m)


@pytest.mark.parametrize("m", [1, 6, 40, 140, 300])
def test_the_largest_sums(native, m):
    """All codes -128 at the largest k: the sum is 2^14 k, just inside 32 bits; and its negative with 127."""
    n, k = 40, 131040
    one, xs = torch.ones(n), torch.ones(m)
    x = torch.full((m, k), -128, dtype=torch.int8)
    for v in (-128, 127):
        w = torch.full((n, k), v, dtype=torch.int8)
        y = native.ffn_int8_linear(x.cuda(), w.cuda(), one.cuda(), x_scales=xs.cuda())
        assert torch.all(y.float().cpu() == torch.tensor(float(-128 * v * k)).to(torch.bfloat16).float())


@pytest.mark.parametrize("m,n,k", [(1, 1000, 1056), (4, 256, 4096), (37, 1000, 1056), (90, 96, 640), (300, 520, 1056)])
def test_linear_of_bf16_rows_quantises_them_first(native, m, n, k):
    x, w, ws = rows(m, k, 5).cuda(), codes(n, k, 6).cuda(), scales(n, k, 7).cuda()
    y = native.ffn_int8_linear(x, w, ws)
    assert same_bits(y, native.ffn_int8_linear(*(lambda c, s: (c, w, ws, s))(*native.ffn_int8_quantize(x))))
    xq, xs = I.quantize_rows(x.float().cpu().numpy())
    assert same_bits(y.cpu(), ref_linear(torch.from_numpy(xq), torch.from_numpy(xs), w.cpu(), ws.cpu()))


def test_a_quantised_weight(native):
    w, x = rows(300, 672, 8), rows(21, 672, 9)
    wq, ws = native.ffn_int8_quantize(w.cuda())
    y = native.ffn_int8_linear(x.cuda(), wq, ws)
    # each factor is off by at most half a step of its row: |y - y64| <= sum |x| step_w / 2 + |w| step_x / 2 + both, then bf16
    x64, w64 = x.double().numpy(), w.double().numpy()
    sx, sw = np.abs(x64).max(1)[:, None] / 127, np.abs(w64).max(1)[None, :] / 127
    ref = x64 @ w64.T
    bound = np.abs(x64).sum(1)[:, None] * sw / 2 + np.abs(w64).sum(1)[None, :] * sx / 2 + 672 * sx * sw / 4
    assert np.all(np.abs(bf16_to_f64(y) - ref) <= 1.001 * bound + 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("n,k", [(1000, 1056), (256, 4096), (96, 64)])
def test_rows_do_not_depend_on_the_batch(native, n, k):
    x, w, ws = rows(700, k, 10).cuda(), codes(n, k, 11).cuda(), scales(n, k, 12).cuda()
    whole = native.ffn_int8_linear(x, w, ws)
    for m in (1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 512):
        assert same_bits(native.ffn_int8_linear(x[:m].contiguous(), w, ws), whole[:m]), m


@pytest.mark.parametrize("m", [1, 5, 30, 100, 200, 300])
@pytest.mark.parametrize("n", [72, 1001])
def test_only_its_rows_are_written(native, m, n):
    k = 160
    y = torch.full((m + 3, n), 9.0, dtype=torch.bfloat16, device="cuda")
    x, w, ws = rows(m, k, 13).cuda(), codes(n, k, 14).cuda(), scales(n, k, 15).cuda()
    native.ffn_int8_linear(x, w, ws, y=y[:m])
    torch.cuda.synchronize()
    assert torch.all(y[m:] == 9) and not torch.any(torch.isnan(y[:m]))
    native.ffn_int8_linear(x[:0], w, ws, y=y[:0])
    assert native.ffn_int8_forward(x[:0], codes(2 * 96, k, 1).cuda(), scales(192, k, 1).cuda(), codes(k, 96, 2).cuda(),
                                   scales(k, 96, 2).cuda()).shape == (0, k)


@pytest.mark.parametrize("m", [2, 40, 140, 300])
def test_rows_of_nan_stay_by_themselves(native, m):
    x, w, ws = rows(m, 224, 16), codes(100, 224, 17).cuda(), scales(100, 224, 18).cuda()
    good = native.ffn_int8_linear(x.cuda(), w, ws)
    x[m // 2, 100] = float("nan")
    x[0, 0] = float("inf")
    y = native.ffn_int8_linear(x.cuda(), w, ws)
    assert torch.all(torch.isnan(y[0])) and torch.all(torch.isnan(y[m // 2]))
    keep = [i for i in range(m) if i not in (0, m // 2)]
    assert same_bits(y[keep], good[keep])
    ws2 = ws.clone()
    ws2[7] = float("nan")
    y = native.ffn_int8_linear(x.cuda(), w, ws2)
    assert torch.all(torch.isnan(y[:, 7])) and same_bits(y[keep][:, 8:], good[keep][:, 8:])


# --------------------------------------------------------------------- layer

def layer(hidden, inter, seed):
    return (codes(2 * inter, hidden, seed), scales(2 * inter, hidden, seed + 1), codes(hidden, inter, seed + 2), scales(hidden, inter, seed + 3))


def check_forward(native, x, weights, **kw):
    """Bit for bit where no hidden value is near a rounding.

    A hidden value may be rounded to the other neighbour where the fp32 value may be off by more than its distance from
    the midpoint.  In half steps of fp32 (2^-24 relative): the gate and up products 3 each (sum, two factors), of which
    the gate's enter with at most 1 + |z|; exp 2 (2 + 1.173 |z|), the addition 1, the quotient 4, the product 1: at most
    16 + 6 |z|.  Such a value moves by one bf16 step, at most 2^-7 of the row's largest, and its code, of 1/127 of it, by
    at most one.  Rows whose largest value is so near a midpoint are held to the error of a scale that is off by 2^-7:
    every code may move by one, and all are scaled by 1 + 2^-7."""
    gu, gus, dn, dns = (t.numpy() for t in weights)
    out = native.ffn_int8_forward(x.cuda(), *(t.cuda() for t in weights), **kw)
    torch.cuda.synchronize()
    xq, xs = I.quantize_rows(x.float().numpy())
    g, h = I.hidden_rows(xq, xs, gu, gus)
    hb = np.asarray(O.round_to_bf16(h), dtype=np.float64)
    ulp = bf16_ulp(h)
    with np.errstate(invalid="ignore"):
        from_mid = np.abs(np.abs(np.abs(h) - np.floor(np.abs(h) / ulp) * ulp) - ulp / 2)
    near = from_mid <= (16 + 6 * np.abs(g)) * 2.0 ** -24 * np.abs(h)
    hq, hs = I.quantize_rows(hb)
    v = I.linear(hq, hs, dn, dns).astype(np.float64)
    got, ref = bf16_to_f64(out), torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)
    exact = ~near.any(1)
    assert same_bits(out.cpu()[exact], ref[exact])
    top = np.argmax(np.abs(hb), axis=1)
    a = np.abs(hb).max(1, keepdims=True)
    top_near = np.any(near & (np.abs(hb) >= a * (1 - 2.0 ** -6)), axis=1)
    step = hs[:, None].astype(np.float64) * dns[None, :].astype(np.float64)
    loose = np.where(top_near[:, None], step * np.abs(dn.astype(np.float64)).sum(1)[None, :] * 1.01 + 2.0 ** -7 * np.abs(v), 0.0)
    tight = step * (near.astype(np.float64) @ np.abs(dn.astype(np.float64)).T)
    assert np.all(np.abs(got - v) <= tight + loose + 2.0 ** -8 * np.abs(v) * (1 + 2.0 ** -6) + 2.0 ** -8 * tight), top
    return out, exact


@pytest.mark.parametrize("m,hidden,inter", [(1, 32, 32), (1, 256, 512), (2, 1056, 672), (3, 64, 96), (4, 512, 1024), (5, 96, 1600), (8, 256, 256),
                                            (13, 160, 352), (33, 1056, 672), (64, 128, 96), (70, 256, 480), (129, 352, 128), (150, 96, 1056),
                                            (256, 256, 256), (301, 1056, 672), (520, 512, 416)])
def test_forward(native, m, hidden, inter):
    out, exact = check_forward(native, rows(m, hidden, m + 20), layer(hidden, inter, 21))
    assert m < 20 or exact.sum() > 0


def test_forward_of_quantised_rows_and_into_its_input(native):
    for m in (1, 7, 40, 200, 300):
        x, weights = rows(m, 288, 30).cuda(), [t.cuda() for t in layer(288, 416, 31)]
        out = native.ffn_int8_forward(x, *weights)
        xq, xs = native.ffn_int8_quantize(x)
        assert same_bits(native.ffn_int8_forward(xq, *weights, x_scales=xs), out)
        assert native.ffn_int8_forward(x, *weights, out=x) is x and same_bits(x, out)


def test_forward_rows_do_not_depend_on_the_batch(native):
    x, weights = rows(600, 256, 40).cuda(), [t.cuda() for t in layer(256, 672, 41)]
    whole = native.ffn_int8_forward(x, *weights)
    for m in (1, 2, 4, 5, 8, 9, 16, 17, 48, 64, 65, 128, 129, 200, 256, 257, 512):
        assert same_bits(native.ffn_int8_forward(x[:m].contiguous(), *weights), whole[:m]), m


def test_zero_rows_and_nan_rows_of_the_layer(native):
    for m in (3, 50, 140, 300):
        x, weights = rows(m, 128, 50), [t.cuda() for t in layer(128, 160, 51)]
        good = native.ffn_int8_forward(x.cuda(), *weights)
        x[0], x[1, 5] = 0.0, float("nan")
        out = native.ffn_int8_forward(x.cuda(), *weights)
        assert torch.all(out[0] == 0) and torch.all(torch.isnan(out[1])) and same_bits(out[2:], good[2:])


# -------------------------------------------------- streams, graphs, workspaces

def test_workspaces_of_garbage_and_of_a_larger_batch(native):
    weights = [t.cuda() for t in layer(256, 352, 60)]
    ws = torch.full((native.ffn_int8_workspace_size(300, 256, 352),), 255, dtype=torch.uint8, device="cuda")
    for m in (300, 1, 40, 150, 2, 299):
        x = rows(m, 256, 60 + m).cuda()
        assert same_bits(native.ffn_int8_forward(x, *weights, workspace=ws), native.ffn_int8_forward(x, *weights))
    with pytest.raises(native.FfnError) as e:
        native.ffn_int8_forward(rows(301, 256, 1).cuda(), *weights, workspace=ws)
    assert e.value.status_name == "FFN_ERR_WORKSPACE"


@pytest.mark.parametrize("m", [1, 20, 140, 300])
def test_on_another_stream(native, m):
    weights = [t.cuda() for t in layer(256, 352, 70)]
    x = rows(m, 256, 70).cuda()
    ref = native.ffn_int8_forward(x, *weights)
    ref_lin = native.ffn_int8_linear(x, weights[0], weights[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = native.ffn_int8_forward(x, *weights, stream=side)
    y = native.ffn_int8_linear(x, weights[0], weights[1], stream=side)
    with torch.cuda.stream(side):
        c, s = native.ffn_int8_quantize(x)
        y2 = native.ffn_int8_linear(c, weights[0], weights[1], x_scales=s)
    torch.cuda.current_stream().wait_stream(side)
    assert same_bits(out, ref) and same_bits(y, ref_lin) and same_bits(y2, ref_lin)


@pytest.mark.parametrize("m", [1, 2, 30, 300])
def test_weights_written_right_before_the_call(native, m):
    """A weight that the work ahead in the stream still writes, a kernel of another library or the quantisation here."""
    n, k = 6000, 2048
    x, full, ws = rows(m, k, 75).cuda(), [codes(n, k, 76 + i).cuda() for i in range(2)], scales(n, k, 78).cuda()
    xq, xs = native.ffn_int8_quantize(x)
    refs = [native.ffn_int8_linear(x, w, ws) for w in full]
    big = [rows(n, k, 79 + i).cuda() for i in range(2)]
    quantised = [native.ffn_int8_quantize(b) for b in big]
    refs_q = [native.ffn_int8_linear(x, *q) for q in quantised]
    torch.cuda.synchronize()
    w, c, s = torch.empty_like(full[0]), torch.empty_like(full[0]), torch.empty_like(ws)
    for i in (0, 1, 0, 1):
        w.copy_(full[i])
        y = native.ffn_int8_linear(x, w, ws)
        w.copy_(full[1 - i])
        y2 = native.ffn_int8_linear(xq, w, ws, x_scales=xs)
        native.ffn_int8_quantize(big[i], codes=c, scales=s)
        y3 = native.ffn_int8_linear(xq, c, s, x_scales=xs)
        native.ffn_int8_quantize(big[1 - i], codes=c, scales=s)
        y4 = native.ffn_int8_linear(x, c, s)
        assert same_bits(y, refs[i]) and same_bits(y2, refs[1 - i]) and same_bits(y3, refs_q[i]) and same_bits(y4, refs_q[1 - i])


@pytest.mark.parametrize("m", [1, 20, 140, 300])
def test_two_graphs_that_share_a_workspace(native, m):
    weights = [t.cuda() for t in layer(256, 352, 80)]
    ws = torch.empty((native.ffn_int8_workspace_size(m, 256, 352),), dtype=torch.uint8, device="cuda")
    x1, x2 = rows(m, 256, 81).cuda(), rows(m, 256, 82).cuda()
    o1, o2 = torch.empty_like(x1), torch.empty_like(x2)
    native.ffn_int8_forward(x1, *weights, out=o1, workspace=ws)
    graphs = []
    for x, o in ((x1, o1), (x2, o2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            native.ffn_int8_forward(x, *weights, out=o, workspace=ws)
        graphs.append(g)
    for seed in (83, 84):
        x1.copy_(rows(m, 256, seed))
        x2.copy_(rows(m, 256, seed + 10))
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
        assert same_bits(o1, native.ffn_int8_forward(x1, *weights)) and same_bits(o2, native.ffn_int8_forward(x2, *weights))


def test_many_calls_back_to_back(native):
    """Calls whose kernels overlap by their launch order: each reads what the one before wrote."""
    weights = [t.cuda() for t in layer(256, 256, 90)]
    for m in (1, 24, 140, 260):
        x = rows(m, 256, 91).cuda()
        ws = torch.empty((native.ffn_int8_workspace_size(m, 256, 256),), dtype=torch.uint8, device="cuda")
        a = x
        for _ in range(12):
            a = native.ffn_int8_forward(a, *weights, workspace=ws)
        b = x
        for _ in range(12):
            b = native.ffn_int8_forward(b, *weights)
            torch.cuda.synchronize()
        assert same_bits(a, b)
