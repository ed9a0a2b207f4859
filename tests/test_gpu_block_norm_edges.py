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


#: Rows of every kernel: a warp's, a CTA's, one by one (few, many, long), and the streaming kernel's.
PLACES = [(3, 96), (4, 1000), (5, 2048), (4, 20000), (5, 99), (3, 9001), (1500, 1037), (2100, 384), (700, 2000), (450, 5120)]


def near_constant_error(v, p):
    """norm_error, of a row that has given up its mean.

    What is left of the mean then is at most 128 of the root of the variance and eps (else it is given up once more), so
    its error of 72 half steps is taken of 128 + 1 of them in the place of the mean magnitude.  The subtraction is off by
    half a step of each difference, which is one of norm_error's 48.  Where the mean is not given up it is below 128 too."""
    v = np.asarray(v, dtype=np.float64)
    t = np.abs(I.norm(v, **dict(p, weight=None, bias=None)))
    err = (49 * t + 72 * 129 * (1 + 2 * t)) * (1.0 if p["weight"] is None else np.abs(p["offset"] + p["weight"]))
    return HALF * (err + (0 if p["bias"] is None else 2 * np.abs(p["bias"])))


def check_near_constant(native, r, hidden):
    """fp32 rows as the residual, and, where they are bf16 numbers, as y."""
    n, p = make_norm(native, hidden, "layer", torch.float32, seed=3)
    ref, err = I.norm(r.double().numpy(), **p), near_constant_error(r.double().numpy(), p)
    x = bf16_to_f64(native.ffn_block_norm(r.cuda(), pre=n)[1])
    assert np.all(np.abs(x - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err)), np.nanmax(np.abs(x - ref))
    if torch.equal(r, r.to(torch.bfloat16).float()):
        z = native.ffn_block_norm(torch.zeros_like(r).cuda(), y=r.to(torch.bfloat16).cuda(), post=n)[0].double().cpu().numpy()
        assert np.all(np.abs(z - ref) <= err + HALF * (4 * np.abs(ref) + err)), np.nanmax(np.abs(z - ref))


@pytest.mark.parametrize("m,hidden", PLACES)
def test_layer_norms_of_rows_of_one_value(native, m, hidden):
    """Their bias: the rounding of a mean is not normalised in the place of values."""
    r = rows(m, hidden, 4).to(torch.bfloat16).float()
    for value in (1000.0, -1.1e6, 2.2e10, 1.3e30, -3.3895314e38, 3e-5):
        r[1] = value
        check_near_constant(native, r.to(torch.bfloat16).float(), hidden)
    r[1] = 1234.567  # (not a bf16 number)
    check_near_constant(native, r, hidden)


@pytest.mark.parametrize("m,hidden", PLACES)
def test_layer_norms_of_values_that_hardly_differ(native, m, hidden):
    """A mean of up to 2^23 times what they differ by, neighbouring numbers at the end."""
    g = torch.Generator().manual_seed(hidden)
    r = rows(m, hidden, 4).float()
    for i, ratio in enumerate((100.0, 130.0, 2e3, 1e5, 3e6)):
        r[1:3] = (ratio * torch.randn((2, 1), generator=g, dtype=torch.float64) + torch.randn((2, hidden), generator=g, dtype=torch.float64)).float()
        check_near_constant(native, r, hidden)
    r[1] = torch.where(torch.rand(hidden, generator=g) < 0.5, 1e6, np.float32(np.nextafter(np.float32(1e6), np.float32(2e6))).item())
    check_near_constant(native, r, hidden)


@pytest.mark.parametrize("shapes", [[(600, 2048), (400, 8192)], [(5, 99), (5, 30001)]])
def test_calls_from_several_threads(native, shapes):
    """Rows of different widths through the same kernel at once, each thread on its own stream: each has its shared
    memory whatever the others ask for.  (Two seconds; the C entry itself, so that the calls meet.)"""
    import ctypes
    import threading
    import time
    from test_int8_abi import BlockArgs
    calls = []
    for m, hidden in 2 * shapes:
        r, y = rows(m, hidden, 1).cuda(), rows(m, hidden, 2).cuda()
        n = make_norm(native, hidden, seed=1)[0]
        out, res = torch.empty_like(r), torch.empty_like(r)
        norm = native._norm_now(n, "pre", hidden, 0)[0] if hasattr(native, "_norm_now") else n._address
        a = BlockArgs(y=y.data_ptr(), y_stride=hidden, post=norm, residual=r.data_ptr(), residual_type=1, residual_stride=hidden,
                      residual_out=res.data_ptr(), residual_out_stride=hidden, residual_scale=1.0, branch_scale=1.0, pre=norm,
                      out=out.data_ptr(), out_stride=hidden)
        calls.append((m, hidden, a, (r, y, n, out, res), torch.cuda.Stream(), native.ffn_block_norm(r, y=y, post=n, pre=n)))
    torch.cuda.synchronize()
    until, bad = time.monotonic() + 2, []

    def work(m, hidden, a, keep, stream, first):
        torch.cuda.set_device(0)
        call, at, raw, n = native.lib.ffn_block_norm, ctypes.byref(a), stream.cuda_stream, 0
        while time.monotonic() < until and not bad:
            for _ in range(200):
                status = call(at, m, hidden, raw)
                if status:
                    bad.append((m, hidden, n, status))
                    break
            n += 200
            stream.synchronize()

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    for _, _, _, (_, _, _, out, res), _, first in calls:
        assert same_bits(out, first[1]) and same_bits(res, first[0])


def same_kind(got, ref, scale):
    """Infinities with their signs and NaN in the same places; elsewhere within 2^-6 of the largest factor there."""
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isposinf(got), np.isposinf(ref)) \
        and np.array_equal(np.isneginf(got), np.isneginf(ref))
    ok = np.isfinite(ref)
    assert np.all(np.abs(got[ok] - ref[ok]) <= 2.0 ** -6 * (np.abs(ref[ok]) + scale))


@pytest.mark.parametrize("m,hidden", PLACES)
@pytest.mark.parametrize("post", ["rms", "layer", None])
@pytest.mark.parametrize("gate", ["row", "channel", "full"])
def test_infinite_gates(native, m, hidden, post, gate):
    """Gates, or products with them, that are not finite, whichever kernel takes the rows: an infinity of z's sign, NaN where z is 0."""
    inf, nan = float("inf"), float("nan")
    shape = {"row": (m, 1), "channel": (1, hidden), "full": (m, hidden)}[gate]
    g = torch.randn(shape, generator=torch.Generator().manual_seed(1))
    g.view(-1)[:3] = torch.tensor([inf, -inf, nan if gate != "channel" else 3e38])
    y, r = rows(m, hidden, 2), rows(m, hidden, 3).float()
    y[:, 1::7] = 0.0
    n, p = (None, None) if post is None else make_norm(native, hidden, post, torch.float32, seed=4)
    pre = make_norm(native, hidden, "layer", torch.float32, seed=5)[0]
    res, x = native.ffn_block_norm(r.cuda(), y=y.cuda(), post=n, gate=g.cuda(), pre=pre, branch_scale=0.5)
    with np.errstate(invalid="ignore", over="ignore"):
        z = y.double().numpy() if n is None else I.norm(y.double().numpy(), **p)
        ref = (r.double().numpy() + 0.5 * g.double().numpy() * z).astype(np.float32).astype(np.float64)  # (the residual's type)
    same_kind(res, ref, 8.0)
    bad = ~np.isfinite(ref).all(1)
    assert np.array_equal(np.isnan(x.float().cpu().numpy()).any(1), bad)


@pytest.mark.parametrize("m,hidden", PLACES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["row", "channel", "full"])
def test_large_gates_of_small_values(native, m, hidden, kind, gate):
    """A gate times a norm's factor, 1000 for values far below the root of eps, may pass fp32's range where the product
    with the value does not."""
    shape = {"row": (m, 1), "channel": (1, hidden), "full": (m, hidden)}[gate]
    g = 1e36 * (1 + torch.rand(shape, generator=torch.Generator().manual_seed(1)))
    y, r = (1e-8 * rows(m, hidden, 2).float()).to(torch.bfloat16), 1e30 * rows(m, hidden, 3).float()
    n, p = make_norm(native, hidden, kind, torch.float32, bias=False, seed=4)
    res = native.ffn_block_norm(r.cuda(), y=y.cuda(), post=n, gate=g.cuda(), branch_scale=0.5)[0]
    ref = r.double().numpy() + 0.5 * g.double().numpy() * I.norm(y.double().numpy(), **p)
    assert np.all(np.isfinite(ref.astype(np.float32)))
    same_kind(res, ref, 1e27)


@pytest.mark.parametrize("m,hidden", PLACES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_infinities_in_what_a_norm_reads(native, m, hidden, kind):
    """The formula's course in every kernel: NaN rows, or zeros (and the bias) around the NaN of an infinity."""
    n, p = make_norm(native, hidden, kind, torch.float32, seed=3)
    r = rows(m, hidden, 4).float()
    r[0, 0], r[1, hidden // 2], r[2, hidden - 1] = float("inf"), -float("inf"), float("nan")
    with np.errstate(invalid="ignore"):
        ref = I.norm(r.double().numpy(), **p)
    assert np.isnan(ref[2]).all() and np.isnan(ref[:2]).sum() == (2 if kind == "rms" else 2 * hidden)
    x = native.ffn_block_norm(r.cuda(), pre=n)[1]
    same_kind(x, ref, 2.0 ** -3)
    if hidden % 32 == 0:
        c, s = native.ffn_block_norm(r.cuda(), pre=n, quantize=True)[1:]
        assert torch.isnan(s).nonzero().flatten().tolist() == [0, 1, 2] and torch.all(c[:3] == 0)
    y = r.to(torch.bfloat16)
    z = native.ffn_block_norm(torch.zeros_like(r).cuda(), y=y.cuda(), post=n)[0]
    with np.errstate(invalid="ignore"):
        same_kind(z, I.norm(y.double().numpy(), **p), 2.0 ** -3)


@pytest.mark.parametrize("m,hidden", [(3, 96), (5, 2048), (700, 1024)])
def test_codes_at_any_address(native, m, hidden):
    """Tensors are aligned to their elements, and a code is one byte."""
    r, n = rows(m, hidden, 1).cuda(), make_norm(native, hidden)[0]
    for offset in (1, 4, 8):
        buffer = torch.full((m * hidden + 16,), 55, dtype=torch.int8, device="cuda")
        out = buffer[offset:offset + m * hidden].view(m, hidden)
        c, s = native.ffn_block_norm(r, pre=n, quantize=True, out=out)[1:]
        rc, rs = native.ffn_int8_quantize(native.ffn_block_norm(r.clone(), pre=n)[1])
        assert c is out and torch.all(buffer[:offset] == 55) and torch.all(buffer[offset + m * hidden:] == 55)
        step = rs[:, None] * 127 * 2.0 ** -7 + rs[:, None]  # (sums in another order: a bf16 step, and a code)
        assert torch.all(torch.isfinite(s)) and torch.all((c.float() * s[:, None] - rc.float() * rs[:, None]).abs() <= step)
