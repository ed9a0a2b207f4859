"""Norms around a layer on the GPU against the fp64 oracle, and in their place
between the layers."""
import numpy as np
import pytest
import torch

from oracle import int8 as I
from nvfp4_quantized_dense_w4a16_b200 import synth

pytestmark = pytest.mark.gpu

from gpu_helpers import bf16_to_f64, gpu_weight
from test_gpu_int8 import codes, native, no_device_error, rows, same_bits, scales  # noqa: F401

HALF = 2.0 ** -24  # half a step of fp32


def make_norm(native, hidden, kind="rms", dtype=torch.bfloat16, offset=0.0, bias=True, weight=True, eps=1e-6, seed=0):
    g = torch.Generator().manual_seed(seed + hidden)
    w = (1.0 - offset + 0.3 * torch.randn(hidden, generator=g)).to(dtype) if weight else None
    b = (0.2 * torch.randn(hidden, generator=g)).to(dtype) if bias and kind == "layer" else None
    n = native.Norm(None if w is None else w.cuda(), None if b is None else b.cuda(), kind=kind, offset=offset, eps=eps)
    f64 = lambda t: None if t is None else t.double().numpy()
    return n, dict(weight=f64(w), bias=f64(b), kind=kind, eps=float(np.float32(eps)), offset=float(np.float32(offset)))


def norm_error(v, p):
    """How far an fp32 norm of the exact rows v may be off, in absolute terms.

    In half steps: a thread adds at most 32 terms of a row, then 5 steps in its warp and 32 warps: a sum of squares is off
    by at most 32 + 5 + 32 additions and 1 for its squares, which the root halves; the reciprocal root 4, the mean's share
    and eps 3; the factors and the bias 4: at most 48 of the result, and of the result without the bias.  The layer norm's
    mean is off by 72 half steps of the mean magnitude, which goes over to each difference, and (twice) into the squares."""
    v = np.asarray(v, dtype=np.float64)
    plain = dict(p, weight=None, bias=None)
    t = np.abs(I.norm(v, **plain))
    factor = 1.0 if p["weight"] is None else np.abs(p["offset"] + p["weight"])
    err = 48 * t
    if p["kind"] == "layer":
        d = v - v.mean(1, keepdims=True)
        inv = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + p["eps"])
        err = err + 72 * np.abs(v).mean(1, keepdims=True) * inv * (1 + 2 * t)
    err = err * factor
    return HALF * (err + (0 if p["bias"] is None else 2 * np.abs(p["bias"])))


def half_step(t):
    return 2.0 ** -8 if t == torch.bfloat16 else 2.0 ** -24


def check(native, m, hidden, residual=torch.bfloat16, weight=torch.bfloat16, kind="rms", offset=0.0, branch=True, post=True, pre=True,
          gate="none", activation="none", gate_dtype=torch.bfloat16, a=1.0, b=1.0, seed=0, y=None, r=None, spread=1.0, **kw):
    y = rows(m, hidden, seed + 1) if y is None else y
    r = (3.0 * rows(m, hidden, seed + 2).float() + spread).to(residual) if r is None else r
    n_post, p_post = make_norm(native, hidden, kind, weight, offset, seed=1) if post and branch else (None, None)
    n_pre, p_pre = make_norm(native, hidden, kind, weight, offset, seed=2) if pre else (None, None)
    shape = {"none": None, "row": (m, 1), "channel": (1, hidden), "vector": (hidden,), "full": (m, hidden), "one": (1, 1)}[gate]
    g = None if shape is None else torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(gate_dtype)
    args = dict(post=n_post, gate=None if g is None else g.cuda(), gate_activation=activation, residual_scale=a, branch_scale=b) if branch else {}
    got = native.ffn_block_norm(r.cuda() if not r.is_cuda else r, y=(y.cuda() if not y.is_cuda else y) if branch else None, pre=n_pre, **args, **kw)
    torch.cuda.synchronize()
    r64, y64 = r.double().cpu().numpy(), y.double().cpu().numpy()
    stored = r64
    if branch:
        z = I.norm(y64, **p_post) if post else y64
        g64 = 1.0 if g is None else I.gate_value(g.double().numpy(), activation)
        ref = I.residual(r64, z, None if g is None else g.double().numpy(), activation, a, b)
        # the branch: the norm's error, the gate's function (exp, sum, quotient; tanh: 8 half steps at most, 1 + |g| more for
        # exp's argument is within them for a bounded g), three products; then the sum and the store
        err = (norm_error(y64, p_post) if post else 0.0) * np.abs(g64 * b) + HALF * (12 + 4 * (g is not None)) * np.abs(g64 * z * b) \
            + HALF * (2 * np.abs(a * r64) + 2 * np.abs(ref))
        stored = got[0].double().cpu().numpy()
        assert got[0].dtype == residual
        tol = err + half_step(residual) * (np.abs(ref) + err) + 2.0 ** -133
        assert np.all(np.abs(stored - ref) <= tol), np.max(np.abs(stored - ref) / tol)
    else:
        assert got[0] is r or same_bits(got[0].cpu(), r.cpu())
    if pre:
        ref = I.norm(stored, **p_pre)
        err = norm_error(stored, p_pre)
        x = got[1].double().cpu().numpy()
        tol = err + 2.0 ** -8 * (np.abs(ref) + err) + 2.0 ** -133
        assert np.all(np.abs(x - ref) <= tol), np.max(np.abs(x - ref) / tol)
    else:
        assert got[1] is None
    return got


HIDDEN = [1, 2, 7, 8, 31, 32, 33, 64, 100, 248, 250, 256, 257, 258, 264, 384, 512, 520, 1000, 1024, 1032, 1037, 2046, 2047, 2048, 2049, 2050, 4094, 4096, 4097, 4098, 5120, 8191, 8192, 8194, 8200, 9001, 9002,
          16384, 16392, 20000, 32766, 32768, 32767]


@pytest.mark.parametrize("hidden", HIDDEN)
@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
def test_widths(native, hidden, residual):
    check(native, 5, hidden, residual, gate="full", activation="sigmoid", a=0.9, b=0.5, seed=hidden)


@pytest.mark.parametrize("hidden", [1, 40, 257, 512, 1000, 1037, 5120, 16392])
@pytest.mark.parametrize("weight", [torch.bfloat16, torch.float32])
def test_layer_norms(native, hidden, weight):
    check(native, 6, hidden, torch.float32, weight, "layer", gate="channel", activation="tanh", gate_dtype=torch.float32, seed=hidden, spread=20.0)


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", ["none", "row", "channel", "vector", "full", "one"])
@pytest.mark.parametrize("hidden", [96, 99, 1536, 2051])
def test_combinations(native, post, pre, gate, hidden):
    for kind, offset, act, dtype in (("rms", 1.0, "none", torch.float32), ("layer", 0.0, "tanh", torch.bfloat16)):
        check(native, 9, hidden, post=post, pre=pre, gate=gate, kind=kind, offset=offset, activation=act if gate != "none" else "none", gate_dtype=dtype,
              seed=hidden)


@pytest.mark.parametrize("m", [0, 1, 2, 7, 8, 9, 150, 1000, 20000])
@pytest.mark.parametrize("hidden", [64, 72, 300, 1040])
def test_rows(native, m, hidden):
    check(native, m, hidden, gate="row", activation="sigmoid", seed=m)
    check(native, m, hidden, torch.float32, branch=False, seed=m)


@pytest.mark.parametrize("m,hidden", [(3000, 288), (2100, 384), (1500, 1000), (700, 2048), (601, 2056), (450, 5120), (400, 8192), (310, 12288), (300, 16384)])
@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
def test_many_rows(native, m, hidden, residual):
    """The streaming kernel: rows that fill its groups unevenly, every kind of gate, biases, quantised outputs."""
    check(native, m, hidden, residual, gate="channel", offset=1.0, a=0.9, b=0.5, seed=m)
    check(native, m, hidden, residual, torch.float32, "layer", gate="full", activation="tanh", seed=m, spread=10.0)
    check(native, m, hidden, residual, gate="full", gate_dtype=torch.float32, activation="sigmoid", pre=False, seed=m)
    check(native, m, hidden, residual, gate="row", post=False, kind="layer", seed=m)
    check(native, m, hidden, residual, branch=False, seed=m)
    if hidden % 32 == 0:
        r, y = rows(m, hidden, 4).to(residual).cuda(), rows(m, hidden, 5).cuda()
        post, pre = make_norm(native, hidden, seed=1)[0], make_norm(native, hidden, "layer", seed=2)[0]
        res, x = native.ffn_block_norm(r, y=y, post=post, pre=pre)
        res2, c, s = native.ffn_block_norm(r, y=y, post=post, pre=pre, quantize=True, residual_out=r)
        rc, rs = native.ffn_int8_quantize(x)
        assert same_bits(res, res2) and torch.equal(c, rc) and torch.equal(s, rs)


def test_many_rows_of_extreme_values(native):
    m, hidden = 1500, 640
    r = torch.randn((m, hidden), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    r[::5] *= 1e37
    r[1::5] *= 0.0
    r[2::5] *= 1e-30
    r[3::5] *= 1e19
    for kind in ("rms", "layer"):
        check(native, m, hidden, torch.float32, kind=kind, branch=False, r=r.float())
        check(native, m, hidden, torch.float32, kind=kind, y=r.to(torch.bfloat16), r=rows(m, hidden, 1).float())
    y, r = rows(m, hidden, 2).cuda(), rows(m, hidden, 3).cuda()
    pre, post = make_norm(native, hidden, seed=1)[0], make_norm(native, hidden, seed=2)[0]
    good = native.ffn_block_norm(r, y=y, post=post, pre=pre)
    y[7, 3], r[8, 5], y[1499, 639] = float("nan"), float("nan"), float("inf")
    _, c, s = native.ffn_block_norm(r, y=y, post=post, pre=pre, quantize=True)
    res, x = native.ffn_block_norm(r, y=y, post=post, pre=pre, residual_out=r, out=y)
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    bad[[7, 8, 1499]] = True
    assert torch.all(torch.isnan(x[bad])) and torch.equal(torch.isnan(s), bad) and torch.all(c[bad] == 0)
    assert same_bits(x[~bad], good[1][~bad]) and same_bits(res[~bad], good[0][~bad])


def test_norms_without_weights(native):
    r = rows(4, 320, 3)
    for kind in ("rms", "layer"):
        n = native.Norm(kind=kind, eps=1e-5)
        x = native.ffn_block_norm(r.cuda(), pre=n)[1]
        p = dict(kind=kind, eps=float(np.float32(1e-5)), weight=None, bias=None, offset=0.0)
        ref = I.norm(r.double().numpy(), **p)
        assert np.all(np.abs(bf16_to_f64(x) - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * norm_error(r.double().numpy(), p))


@pytest.mark.parametrize("hidden", [96, 416, 1056, 4096, 9600, 20000])
@pytest.mark.parametrize("branch", [False, True])
def test_quantised_is_the_quantisation_of_the_plain_output(native, hidden, branch):
    hidden -= hidden % 32
    m = 11
    r, y = rows(m, hidden, 4).cuda(), rows(m, hidden, 5).cuda()
    post, pre = make_norm(native, hidden, seed=1)[0], make_norm(native, hidden, "layer", seed=2)[0]
    kw = dict(y=y, post=post, gate=torch.randn(hidden).cuda()) if branch else {}
    res, x = native.ffn_block_norm(r, pre=pre, **kw)
    res2, c, s = native.ffn_block_norm(r, pre=pre, quantize=True, **kw)
    rc, rs = native.ffn_int8_quantize(x)
    assert same_bits(res, res2) and torch.equal(c, rc) and torch.equal(s, rs)
    # and where the rows are not whole 16 bytes (the scalar path)
    odd = torch.empty((m, hidden + 1), dtype=torch.bfloat16, device="cuda")
    odd[:, 1:] = r
    res3, c, s = native.ffn_block_norm(odd[:, 1:], pre=pre, quantize=True, **kw)
    res4, x = native.ffn_block_norm(odd[:, 1:], pre=pre, **kw)
    rc, rs = native.ffn_int8_quantize(x)
    assert same_bits(res3, res4) and torch.equal(c, rc) and torch.equal(s, rs)


@pytest.mark.parametrize("hidden", [64, 1056])
def test_quantised_rows_that_are_not_whole_16_bytes(native, hidden):
    """Tensors at every alignment of an element: accesses of 8, of 2 and of 1 give the same bits."""
    m = 7
    y, r = rows(m, hidden, 20).cuda(), rows(m, hidden, 21).float().cuda()
    pre, post = make_norm(native, hidden, seed=1)[0], make_norm(native, hidden, seed=2)[0]
    ref = native.ffn_block_norm(r, y=y, post=post, pre=pre, quantize=True)
    for off in (1, 2, 3, 4, 6, 8):
        wy, wr = torch.empty((m, hidden + 10), dtype=torch.bfloat16, device="cuda"), torch.empty((m, hidden + 10), device="cuda")
        wy[:, off:off + hidden], wr[:, off:off + hidden] = y, r
        res, c, s = native.ffn_block_norm(wr[:, off:off + hidden], y=wy[:, off:off + hidden], post=post, pre=pre, quantize=True)
        err = (res - ref[0]).abs()
        assert torch.all(err <= 2.0 ** -20 * ref[0].abs() + 2.0 ** -20)  # sums in another order
        x = native.ffn_block_norm(wr[:, off:off + hidden], y=wy[:, off:off + hidden], post=post, pre=pre)[1]
        rc, rs = native.ffn_int8_quantize(x)
        assert torch.equal(c, rc) and torch.equal(s, rs)


@pytest.mark.parametrize("hidden", [64, 77, 1056, 1055])
def test_strides_places_and_what_is_behind_the_rows(native, hidden):
    m, h = 6, hidden
    wide = lambda t, pad, seed: (rows(m, h + pad, seed) * 2).to(t).cuda()
    y, r = wide(torch.bfloat16, 16, 6)[:, 8:8 + h], wide(torch.float32, 9, 7)[:, 9:]
    out = torch.full((m + 2, h + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    res = torch.full((m + 2, h + 3), 7.0, device="cuda")
    check(native, m, h, torch.float32, y=y, r=r, gate="full", out=out[:m, 16:16 + h], residual_out=res[:m, :h])
    assert torch.all(out[m:] == 7) and torch.all(out[:, :16] == 7) and torch.all(out[:, 16 + h:] == 7)
    assert torch.all(res[m:] == 7) and torch.all(res[:, h:] == 7)
    g = torch.randn((2 * m, h + 1), device="cuda")[::2, 1:]  # a strided gate
    pre = make_norm(native, h)[0]
    a, b = native.ffn_block_norm(r, y=y, gate=g, pre=pre), native.ffn_block_norm(r, y=y, gate=g.contiguous(), pre=pre)
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])


@pytest.mark.parametrize("hidden", [64, 77, 1024, 1055, 5120, 20000])
@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
def test_in_place(native, hidden, residual):
    m = 300
    r, y = rows(m, hidden, 8).to(residual).cuda(), rows(m, hidden, 9).cuda()
    post, pre = make_norm(native, hidden, seed=1)[0], make_norm(native, hidden, seed=2)[0]
    ref = native.ffn_block_norm(r, y=y, post=post, pre=pre, residual_scale=0.5)
    only = native.ffn_block_norm(r, y=y, post=post, pre=pre, residual_scale=0.5, store_residual=False)
    assert only[0] is None and same_bits(only[1], ref[1])
    got = native.ffn_block_norm(r, y=y, post=post, pre=pre, residual_scale=0.5, residual_out=r, out=y)
    assert got[0] is r and got[1] is y and same_bits(r, ref[0]) and same_bits(y, ref[1])


@pytest.mark.parametrize("hidden", [40, 333, 2048])
def test_values_at_the_ends_of_the_range(native, hidden):
    """Squares that pass fp32's range, rows of zeros and of tiny values."""
    big = torch.randn((5, hidden), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    big[0] *= 1e38 / big[0].abs().max()
    big[1] *= 1e30
    big[2] *= 0.0
    big[3] *= 1e-30
    big[4] *= 1e19
    for kind in ("rms", "layer"):
        check(native, 5, hidden, torch.float32, kind=kind, branch=False, r=big.float())
        check(native, 5, hidden, torch.float32, kind=kind, y=big.to(torch.bfloat16), r=rows(5, hidden, 1).float())


def test_nan_and_infinity(native):
    m, h = 5, 416
    r, y = rows(m, h, 10), rows(m, h, 11)
    pre, post = make_norm(native, h, seed=1)[0], make_norm(native, h, seed=2)[0]
    good = native.ffn_block_norm(r.cuda(), y=y.cuda(), post=post, pre=pre)
    y[1, 3] = float("nan")
    y[2, 5] = float("inf")
    r[3, 7] = float("nan")
    res, x = native.ffn_block_norm(r.cuda(), y=y.cuda(), post=post, pre=pre)
    assert torch.all(torch.isnan(x[1])) and torch.all(torch.isnan(x[2])) and torch.all(torch.isnan(x[3]))
    assert torch.all(torch.isnan(res[1])) and torch.isnan(res[2, 5]) and torch.isnan(res[3]).sum() == 1
    assert same_bits(x[[0, 4]], good[1][[0, 4]]) and same_bits(res[[0, 4]], good[0][[0, 4]])
    _, c, s = native.ffn_block_norm(r.cuda(), y=y.cuda(), post=post, pre=pre, quantize=True)
    assert torch.isnan(s).tolist() == [False, True, True, True, False] and torch.all(c[1:4] == 0)


def test_refusals_in_python(native):
    r, y = rows(4, 64, 1).cuda(), rows(4, 64, 2).cuda()
    n = native.Norm(torch.ones(64, device="cuda"))
    call = native.ffn_block_norm
    for kw, what in ((dict(y=y[:3]), "y must"), (dict(y=y[:, :32]), "y must"), (dict(gate=torch.ones(3, 64, device="cuda"), y=y), "gate must"),
                     (dict(y=y, gate_activation="relu"), "gate_activation must"), (dict(out=y), "needs the norm"), (dict(quantize=True), "needs the norm"),
                     (dict(pre=n, out_scales=torch.ones(4, device="cuda")), "needs quantize"), (dict(pre=n, residual_out=r), "needs y"),
                     (dict(pre=native.Norm(torch.ones(32, device="cuda"))), "32 weights"), (dict(y=y, residual_out=r, store_residual=False), "store_residual"),
                     (dict(y=y, pre=n, out=y.t()), "out must")):
        with pytest.raises(ValueError, match=what):
            call(r, **kw)
    for kw in (dict(y=y.float()), dict(y=y, gate=torch.ones(64, device="cuda").double()), dict(pre=torch.ones(64, device="cuda"))):
        with pytest.raises(TypeError):
            call(r, **kw)
    for kw in (dict(), dict(pre=n, residual_scale=0.5), dict(pre=n, gate=y), dict(pre=n, post=n), dict(y=y, store_residual=False),
               dict(y=y, branch_scale=float("nan")), dict(pre=native.Norm(eps=0.0))):
        with pytest.raises(native.FfnError, match="INVALID_ARG"):
            call(r, **kw)
    with pytest.raises(native.FfnError, match="UNSUPPORTED"):
        call(torch.ones((2, 32776), device="cuda"), pre=native.Norm())
    with pytest.raises(native.FfnError, match="SHAPE"):
        call(rows(2, 40, 1).cuda(), pre=native.Norm(), quantize=True)
    with pytest.raises(ValueError, match="one length"):
        native.Norm(torch.ones(4, device="cuda"), torch.ones(5, device="cuda"))


def test_another_stream_and_graphs(native):
    m, h = 30, 1056
    r, y = rows(m, h, 12).cuda(), rows(m, h, 13).cuda()
    post, pre = make_norm(native, h, seed=1)[0], make_norm(native, h, seed=2)[0]
    ref = native.ffn_block_norm(r, y=y, post=post, pre=pre)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = native.ffn_block_norm(r, y=y, post=post, pre=pre, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert same_bits(got[0], ref[0]) and same_bits(got[1], ref[1])
    res, x = torch.empty_like(r), torch.empty_like(r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.ffn_block_norm(r, y=y, post=post, pre=pre, residual_out=res, out=x)
    r.copy_(rows(m, h, 14))
    g.replay()
    ref = native.ffn_block_norm(r, y=y, post=post, pre=pre)
    assert same_bits(res, ref[0]) and same_bits(x, ref[1])


# ------------------------------------------------------------ layers in their blocks

@pytest.mark.parametrize("m", [1, 7, 40, 140, 300])
def test_blocks_of_int8_layers(native, m):
    """Three blocks in a row, norms and quantisation fused, against the same steps one by one with copies between."""
    hidden, inter = 288, 416
    weights = [[codes(2 * inter, hidden, 7 * i), scales(2 * inter, hidden, 7 * i + 1), codes(hidden, inter, 7 * i + 2), scales(hidden, inter, 7 * i + 3)]
               for i in range(3)]
    weights = [[t.cuda() for t in w] for w in weights]
    pres = [make_norm(native, hidden, seed=10 + i)[0] for i in range(4)]
    posts = [make_norm(native, hidden, seed=20 + i)[0] for i in range(3)]
    gates = [torch.randn(hidden, generator=torch.Generator().manual_seed(i)).cuda() for i in range(3)]
    r0 = (2 * rows(m, hidden, 15)).float().cuda()

    r = r0.clone()
    c, s = native.ffn_block_norm(r, pre=pres[0], quantize=True)[1:]
    for i in range(3):
        y = native.ffn_int8_forward(c, *weights[i], x_scales=s)
        last = i == 2
        got = native.ffn_block_norm(r, y=y, post=posts[i], gate=gates[i], gate_activation="tanh", pre=pres[i + 1], quantize=not last, residual_out=r,
                                    **({} if last else dict(out=c, out_scales=s)))
    fused_r, fused_x = r, got[1]

    r = r0
    for i in range(3):
        x = native.ffn_block_norm(r, pre=pres[i])[1]
        torch.cuda.synchronize()
        y = native.ffn_int8_forward(x, *weights[i])
        torch.cuda.synchronize()
        r = native.ffn_block_norm(r, y=y, post=posts[i], gate=gates[i], gate_activation="tanh")[0]
        torch.cuda.synchronize()
    assert same_bits(fused_r, r) and same_bits(fused_x, native.ffn_block_norm(r, pre=pres[3])[1])
    assert torch.all(torch.isfinite(r))


@pytest.mark.parametrize("m", [1, 5, 70])
def test_a_block_of_an_nvfp4_layer(native, m):
    """norm -> ffn_nvfp4_forward -> norm, gate, residual, norm: what the calls one by one give."""
    hidden, inter = 256, 384
    gate = gpu_weight(native, synth.random_bf16((inter, hidden), 1, std=0.05))[0]
    up = gpu_weight(native, synth.random_bf16((inter, hidden), 2, std=0.05))[0]
    down = gpu_weight(native, synth.random_bf16((hidden, inter), 3, std=0.05))[0]
    gate_up = native.ffn_nvfp4_weight_create_gate_up(gate, up)
    r = rows(m, hidden, 16).cuda()
    pre, post = make_norm(native, hidden, seed=1)[0], make_norm(native, hidden, seed=2)[0]
    x = native.ffn_block_norm(r, pre=pre)[1]
    y = native.ffn_nvfp4_forward(x, gate_up, down)
    res, nxt = native.ffn_block_norm(r, y=y, post=post, pre=pre)
    torch.cuda.synchronize()
    y2 = native.ffn_nvfp4_forward(x.clone(), gate_up, down)
    torch.cuda.synchronize()
    assert same_bits(y, y2)
    p = make_norm(native, hidden, seed=2)[1]
    ref = I.residual(r.double().cpu().numpy(), I.norm(bf16_to_f64(y2), **p))
    err = norm_error(bf16_to_f64(y2), p) + HALF * 16 * np.abs(ref)
    assert np.all(np.abs(bf16_to_f64(res) - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err))
    assert same_bits(nxt, native.ffn_block_norm(res, pre=pre)[1])
