"""Rotary positions: frequencies against the published formulas, the rotation and its gradient against 64 bits, and
what the calls refuse.

Tolerance of an output element y = m (x1 cos a -+ x2 sin a): the kernel's float32 error is below 12 half steps of
float32 on m (|x1| + |x2|) (the reduced angle in half turns is rounded once, 2^-25 * pi; sinpi and cospi are good to
a unit in the last place, 2^-23 absolute at most; m, the product and the fused sum round once each), and the result is
rounded once to its type."""
import ctypes as C
import math

import pytest
import torch

import kv_cache_retrieval_b200 as hhr
from kv_cache_retrieval_b200 import build as kbuild

FAKE = 1 << 20
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


# ---------------------------------------------------------------- frequencies (host)

def _formula(rot, base, kind, factor, orig, low, high):
    out = []
    for j in range(rot // 2):
        f = base ** (-2.0 * j / rot)
        if kind == "linear":
            f /= factor
        elif kind == "ntk":
            f = (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * j / rot)
        elif kind == "yarn":
            def dim(t):
                return rot * math.log(orig / (2 * math.pi * t)) / (2 * math.log(base))
            lo, hi = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot // 2 - 1)
            s = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - s) + f / factor * s
        elif kind == "bands":
            s = min(max((orig * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = f / factor * (1 - s) + f * s
        out.append(f)
    return out


@pytest.mark.parametrize("rot", [2, 4, 64, 96, 128])
@pytest.mark.parametrize("kind,factor,orig,low,high", [
    ("none", 1.0, 0, 0, 0), ("linear", 4.0, 0, 0, 0), ("ntk", 8.0, 0, 0, 0), ("yarn", 4.0, 32768, 1.0, 32.0),
    ("yarn", 1.0, 4096, 1.0, 32.0), ("bands", 8.0, 8192, 1.0, 4.0)])
def test_frequencies_follow_the_formulas(rot, kind, factor, orig, low, high):
    if kind == "ntk" and rot == 2:
        return
    kw = dict(low=low, high=high) if kind in ("yarn", "bands") else {}
    f, m = hhr.rope_freqs(rot, base=500000.0, scaling=kind, factor=factor, orig=orig, device="cpu", **kw)
    want = torch.tensor(_formula(rot, 500000.0, kind, factor, orig, low, high), dtype=torch.float64)
    assert f.dtype == torch.float64 and f.shape == (rot // 2,)
    assert torch.allclose(f, want, rtol=1e-13, atol=0)
    assert m == pytest.approx(0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0, rel=2 ** -23)


def test_frequency_defaults_of_the_ramps():
    a, _ = hhr.rope_freqs(128, base=1e4, scaling="bands", factor=8.0, orig=8192, device="cpu")
    b, _ = hhr.rope_freqs(128, base=1e4, scaling="bands", factor=8.0, orig=8192, low=1.0, high=4.0, device="cpu")
    assert torch.equal(a, b)
    assert a[0] == 1.0 and a[-1] == pytest.approx(1e4 ** (-126 / 128) / 8, rel=1e-13)


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=3), dict(rot=-2), dict(base=1.0), dict(base=float("nan")), dict(scaling="linear", factor=0.5),
    dict(scaling="linear", factor=float("inf")), dict(scaling="yarn", factor=2.0, orig=0),
    dict(scaling="bands", factor=2.0, orig=4096, low=4.0, high=4.0), dict(rot=2, scaling="ntk", factor=2.0)])
def test_frequency_refusals(kw):
    args = dict(rot=64, base=1e4, device="cpu")
    args.update(kw)
    with pytest.raises(hhr.HhrError) as e:
        hhr.rope_freqs(args.pop("rot"), **args)
    assert e.value.status == hhr.HHR_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        hhr.rope_freqs(64, scaling="other", device="cpu")


# ---------------------------------------------------------------- refusals (host)

def _call(T=4, H=2, d=64, type=0, rot=64, flags=0, mscale=1.0, freqs=FAKE, pos=FAKE, x=FAKE, xt=128, xh=64, y=2 * FAKE,
          yt=128, yh=64):
    r = hhr.hhr_rotation(rot, flags, mscale)
    return hhr.lib().hhr_rope(T, H, d, type, C.byref(r), freqs, pos, x, xt, xh, y, yt, yh, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(H=-1), 1), (dict(d=0), 1), (dict(d=63), 1), (dict(d=514, yt=2048, yh=514), 2), (dict(type=3), 1),
    (dict(type=7), 1), (dict(rot=3), 1), (dict(rot=66), 1), (dict(rot=-2), 1), (dict(flags=4), 1),
    (dict(mscale=float("nan")), 1), (dict(freqs=None), 1), (dict(freqs=FAKE + 4), 1), (dict(pos=None), 1),
    (dict(pos=FAKE + 2), 1), (dict(x=None), 1), (dict(y=None), 1), (dict(x=FAKE + 1), 1), (dict(xt=-1), 1),
    (dict(yh=-1), 1), (dict(yh=63), 1), (dict(yt=127), 1), (dict(yt=0), 1), (dict(y=FAKE, yt=256), 1),
    (dict(T=1 << 30, H=4, yt=1024), 2)])
def test_rope_refusals(kw, status):
    assert _call(**kw) == status


def test_rope_of_nothing_is_ok():
    assert _call(T=0, x=None, y=None, pos=None) == hhr.HHR_OK
    assert _call(H=0) == hhr.HHR_OK
    r = hhr.lib().hhr_rope(4, 2, 64, 0, None, FAKE, FAKE, FAKE, 128, 64, FAKE, 128, 64, None)
    assert r == hhr.HHR_ERR_INVALID_ARG


def test_python_checks():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hhr.rope(x, torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))   # not on a CUDA device


# ---------------------------------------------------------------- against 64 bits

def exact(x, pos, freqs, mscale=1.0, interleaved=False, transpose=False):
    """(y, m (|x1| + |x2|) widened for the angle's own rounding) in float64 on the CPU."""
    x, pos, freqs = x.detach().double().cpu(), pos.double().cpu(), freqs.cpu()
    n = freqs.numel()
    a = pos[:, None, None] * freqs
    c, s = mscale * torch.cos(a), mscale * torch.sin(a) * (-1.0 if transpose else 1.0)
    y, mag = x.clone(), torch.zeros_like(x)
    i = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x1, x2 = x[..., i[0]], x[..., i[1]]
    y[..., i[0]], y[..., i[1]] = x1 * c - x2 * s, x2 * c + x1 * s
    # per half step of float32; the float64 angle (two products and a rounded 1 / 2 pi in the kernel, one
    # product here) adds 2^-51 |a|
    both = abs(mscale) * (x1.abs() + x2.abs()) * (1 + a.abs() * 2.0 ** -51 / (12 * 2.0 ** -24))
    mag[..., i[0]], mag[..., i[1]] = both, both
    return y, mag


def check(got, x, pos, freqs, **kw):
    y, mag = exact(x, pos, freqs, **kw)
    tol = HALF[got.dtype] * y.abs() + 12 * 2.0 ** -24 * mag * (1 + HALF[got.dtype])
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25          # half a step of its subnormals
    err = (got.double().cpu() - y).abs()
    assert bool((err <= tol).all()), f"worst {float((err / (tol + 1e-300)).max())} of the tolerance"


def _x(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float64).to(dtype).cuda()


def _freqs(rot, base=500000.0):
    return hhr.rope_freqs(rot, base=base)[0] if rot else torch.empty(0, dtype=torch.float64, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,d,rot", [
    (1, 1, 2, 2), (1, 40, 128, 128), (7, 3, 64, 32), (5, 5, 96, 96), (33, 1, 128, 64), (257, 4, 80, 40), (3, 2, 6, 4),
    (9, 7, 512, 512), (1100, 1, 2, 2), (4, 3, 64, 0), (1000, 40, 128, 128), (313, 17, 256, 64), (2500, 5, 34, 34),
    (601, 3, 272, 272)])
def test_rotation(T, H, d, rot, dtype, interleaved):
    x, f = _x((T, H, d), dtype), _freqs(rot)
    pos = torch.randint(0, 1 << 20, (T,), dtype=torch.int32, device="cuda")
    y = hhr.rope(x, pos, f, interleaved=interleaved, mscale=1.25)
    check(y, x, pos, f, mscale=1.25, interleaved=interleaved)


@pytest.mark.gpu
def test_far_and_negative_positions():
    x, f = _x((6, 2, 128), torch.float32), _freqs(128)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 24], dtype=torch.int32, device="cuda")
    check(hhr.rope(x, pos, f), x, pos, f)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("view", ["fused", "heads_first", "odd_start", "every_other", "broadcast", "gapped_elements"])
def test_strides(view, dtype):
    T, H, d = 37, 5, 64
    if view == "fused":
        x = _x((T, H + 4, d), dtype)[:, 2:2 + H]
    elif view == "heads_first":
        x = _x((H, T, d), dtype).transpose(0, 1)
    elif view == "odd_start":
        x = _x((T * H * d + 1,), dtype)[1:].view(T, H, d)
    elif view == "every_other":
        x = _x((2 * T, H, d + 2), dtype)[::2, :, :d]
    elif view == "broadcast":
        x = _x((T, 1, d), dtype).expand(T, H, d)
    else:
        x = _x((T, H, 2 * d), dtype)[..., ::2]
    f, pos = _freqs(d), torch.arange(1000, 1000 + T, dtype=torch.int32, device="cuda")
    check(hhr.rope(x, pos, f), x, pos, f)
    # the same into a strided output whose other elements stay as they were
    room = torch.full((T, H + 3, d + 8), 7.0, dtype=dtype, device="cuda")
    out = room[:, 1:1 + H, 4:4 + d]
    got = hhr.rope(x, pos, f, out=out)
    assert got is out
    check(out.clone(), x, pos, f)
    out.fill_(7.0)
    assert bool((room == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 30])
def test_in_place(rot, interleaved):
    x, f = _x((200, 6, 64), torch.bfloat16), _freqs(rot)
    pos = torch.arange(200, dtype=torch.int32, device="cuda")
    before = x.clone()
    assert hhr.rope(x, pos, f, interleaved=interleaved, out=x) is x
    check(x, before, pos, f, interleaved=interleaved)
    assert torch.equal(x[..., rot:], before[..., rot:])


@pytest.mark.gpu
def test_empty():
    f = _freqs(64)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    assert hhr.rope(_x((0, 3, 64), torch.float16), pos, f).shape == (0, 3, 64)
    one = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert hhr.rope(_x((5, 0, 64), torch.float16), one, f).shape == (5, 0, 64)


# ---------------------------------------------------------------- gradients

@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_gradient_is_the_transposed_rotation(dtype, interleaved):
    T, H, d, rot = 61, 3, 64, 48
    x, g, f = _x((T, H, d), dtype), _x((T, H, d), dtype, 1), _freqs(rot)
    pos = torch.randint(0, 1 << 18, (T,), dtype=torch.int32, device="cuda")
    x.requires_grad_()
    y = hhr.rope(x, pos, f, interleaved=interleaved, mscale=0.75)
    y.backward(g)
    check(x.grad, g, pos, f, mscale=0.75, interleaved=interleaved, transpose=True)


@pytest.mark.gpu
def test_gradient_against_differences():
    """rope is linear, so a difference over any step is exact but for rounding: <g, rope(x + h) - rope(x)> = <grad, h>."""
    T, H, d = 17, 2, 32
    x, g, h = (_x((T, H, d), torch.float32, i) for i in range(3))
    f = _freqs(32)
    pos = torch.arange(5, 5 + T, dtype=torch.int32, device="cuda")
    leaf = x.clone().requires_grad_()
    hhr.rope(leaf, pos, f, interleaved=True).backward(g)
    diff = hhr.rope(x + h, pos, f, interleaved=True).double() - hhr.rope(x, pos, f, interleaved=True).double()
    a, b = float((g.double() * diff).sum()), float((leaf.grad.double() * h.double()).sum())
    # each of the T H d products carries float32 errors of at most 2 x 13 half steps on values of a few units
    bound = 40 * 2.0 ** -24 * float((g.abs() * (x.abs() + h.abs() + 1) * 2).double().sum())
    assert abs(a - b) <= bound


@pytest.mark.gpu
def test_gradient_of_a_broadcast_input_and_an_expanded_gradient():
    T, H, d = 9, 4, 64
    x, f = _x((T, 1, d), torch.float32).requires_grad_(), _freqs(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    hhr.rope(x.expand(T, H, d), pos, f).sum().backward()
    one, _ = exact(torch.ones(T, 1, d), pos, f, transpose=True)
    err = (x.grad.double().cpu() - H * one).abs().max()
    assert float(err) <= H * 2 * 16 * 2.0 ** -24 * 2


@pytest.mark.gpu
def test_out_has_no_gradient():
    x, f = _x((2, 2, 64), torch.float32).requires_grad_(), _freqs(64)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        hhr.rope(x, pos, f, out=torch.empty_like(x))
    with torch.no_grad():
        hhr.rope(x, pos, f, out=torch.empty_like(x))


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_second_derivative(interleaved):
    """The gradient is linear in the incoming one: its gradient for it is the rotation."""
    x, f = _x((5, 2, 64), torch.float32).requires_grad_(), _freqs(48)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    g, h = _x((5, 2, 64), torch.float32, 1).requires_grad_(), _x((5, 2, 64), torch.float32, 2)
    (dx,) = torch.autograd.grad(hhr.rope(x, pos, f, interleaved=interleaved), x, g, create_graph=True)
    (dg,) = torch.autograd.grad(dx, g, h)
    check(dg, h, pos, f, interleaved=interleaved)


# ---------------------------------------------------------------- streams and graphs

@pytest.mark.gpu
def test_captured_forward_and_backward():
    T, H, d = 130, 4, 64
    x, g, f = _x((T, H, d), torch.float32), _x((T, H, d), torch.float32, 1), _freqs(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            leaf = x.detach().requires_grad_()
            torch.autograd.grad(hhr.rope(leaf, pos, f), leaf, g)
    torch.cuda.current_stream().wait_stream(side)
    del leaf
    graph = torch.cuda.CUDAGraph()
    leaf = x.detach().requires_grad_()
    with torch.cuda.graph(graph):
        y = hhr.rope(leaf, pos, f)
        (dx,) = torch.autograd.grad(y, leaf, g)
    for seed in (5, 6):
        with torch.no_grad():
            leaf.copy_(_x((T, H, d), torch.float32, seed))
            pos.add_(1000)
        graph.replay()
        torch.cuda.synchronize()
        check(y.detach(), leaf, pos, f)
        check(dx, g, pos, f, transpose=True)


@pytest.mark.gpu
def test_on_a_side_stream():
    x, f = _x((500, 8, 128), torch.bfloat16), _freqs(128)
    pos = torch.arange(500, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = hhr.rope(x, pos, f)
    side.synchronize()
    check(y, x, pos, f)


@pytest.mark.gpu
def test_python_argument_checks_on_the_gpu():
    x, f = _x((4, 2, 64), torch.bfloat16), _freqs(64)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(positions=pos.long()), dict(positions=pos[:3]), dict(freqs=f.float()), dict(positions=pos.cpu()),
                dict(out=torch.empty(4, 2, 32, dtype=x.dtype, device="cuda")), dict(freqs=f.repeat(2)[::2]),
                dict(out=torch.empty(4, 2, 64, device="cuda"))):
        args = dict(positions=pos, freqs=f)
        args.update(bad)
        with pytest.raises(ValueError):
            hhr.rope(x, args.pop("positions"), args.pop("freqs"), **args)
    with pytest.raises(ValueError):
        hhr.rope(x.double(), pos, f)
    with pytest.raises(hhr.HhrError):
        hhr.rope(x, pos, f.repeat(2))       # 128 of 64 elements
    with pytest.raises(hhr.HhrError):       # rows of the output share elements
        hhr.rope(x, pos, f, out=torch.empty(4, 1, 64, dtype=x.dtype, device="cuda").expand(4, 2, 64))
