"""Rotary positions on torch tensors: frequencies and the differentiable rotation."""
from __future__ import annotations

import ctypes as C

import torch
from torch.autograd import forward_ad

from . import _binding as B

_TYPES = {torch.bfloat16: B.HHR_TYPE_BF16, torch.float16: B.HHR_TYPE_F16, torch.float32: B.HHR_TYPE_F32}
_KINDS = {"none": B.HHR_ROPE_SCALE_NONE, "linear": B.HHR_ROPE_SCALE_LINEAR, "ntk": B.HHR_ROPE_SCALE_NTK,
          "yarn": B.HHR_ROPE_SCALE_YARN, "bands": B.HHR_ROPE_SCALE_BANDS}
_TURNS = {"yarn": (1.0, 32.0), "bands": (1.0, 4.0)}   # the published low / high turns


def rope_freqs(rot, base=10000.0, scaling="none", factor=1.0, orig=0, low=None, high=None, device="cuda"):
    """(freqs, mscale): float64 tensor [rot/2] of radians per position on `device`, and the factor on the
    rotated elements.  scaling: "none", "linear", "ntk", "yarn" or "bands" (include/hhr.h, hhr_rope_freqs)."""
    if scaling not in _KINDS:
        raise ValueError(f"scaling must be one of {sorted(_KINDS)}, got {scaling!r}")
    lo, hi = _TURNS.get(scaling, (0.0, 0.0))
    spec = B.hhr_rope_scaling(_KINDS[scaling], orig, base, factor, lo if low is None else low,
                              hi if high is None else high)
    f, mscale = B.hhr_rope_freqs(spec, rot)
    return torch.tensor(f, dtype=torch.float64, device=device), mscale


def on_device(index, fn, *args):
    """Status of fn(*args, stream) on CUDA device `index` with torch's current stream of it."""
    if index < 0:
        raise ValueError("the buffers are not on a CUDA device: the library's kernels need one")
    if index == torch.cuda.current_device():
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(index):
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))


def check_vector(name, t, dtype, length, index):
    """t: contiguous [length] of dtype on CUDA device `index`."""
    if t.dtype is not dtype or t.shape != (length,) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} [{length}] on cuda:{index}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def fits(*sizes):
    """The sizes, which the library takes as int32: ctypes would drop the bits beyond."""
    if max(sizes) >> 31 > 0:
        raise ValueError(f"sizes of 2^31 and more: {sizes}")
    return sizes


# Tells autograd that the library writes the tensors of a tuple: a graph that saved one of them for its gradient then says
# so, instead of taking what it holds by now.  (autograd.graph.increment_version without its own look at the argument.)
written = torch._C._increment_version


_rotations = {}


def rotation(rot, flags, mscale):
    """A reference to an hhr_rotation (kept by value: the few a program uses are made once)."""
    mscale = float(mscale)    # a tensor would be its own key, whatever it holds by then
    r = _rotations.get((rot, flags, mscale))
    if r is None:
        if len(_rotations) >= 64:
            _rotations.clear()
        r = _rotations[rot, flags, mscale] = C.byref(B.hhr_rotation(rot, flags, mscale))
    return r


def _rotate(x, positions, freqs, flags, mscale, out):
    T, H, d = x.shape
    sx, so = x.stride(), out.stride()
    if sx[2] != 1 and d > 1:
        x = x.contiguous()
        sx = x.stride()
    if T >> 31 or H >> 31:
        fits(T, H)
    st = on_device(x.get_device(), B.lib().hhr_rope, T, H, d, _TYPES[x.dtype], rotation(2 * freqs.shape[0], flags, mscale),
                   freqs.data_ptr(), positions.data_ptr(), x.data_ptr(), sx[0], sx[1], out.data_ptr(), so[0], so[1])
    if st:
        raise B.HhrError(st, "hhr_rope")
    return out


def _followed(x):
    """Whether a derivative of x is asked for: a gradient, or the tangent of a dual tensor."""
    return (x.requires_grad and torch.is_grad_enabled()) or \
        (forward_ad._current_level >= 0 and forward_ad.unpack_dual(x).tangent is not None)


def _turn(x, positions, freqs, flags, mscale):
    """x rotated, with the derivatives that are asked for."""
    if _followed(x):
        return _Rope.apply(x, positions, freqs, flags, mscale)
    return _rotate(x, positions, freqs, flags, mscale, x.new_empty(x.shape))


class _Rope(torch.autograd.Function):
    # The rotation is linear: the tangent is the rotation of x's tangent, the gradient the transposed rotation, and the
    # derivatives of these are again the two.
    @staticmethod
    def forward(ctx, x, positions, freqs, flags, mscale):
        ctx.save_for_backward(positions, freqs)
        ctx.save_for_forward(positions, freqs)
        ctx.how = flags, mscale
        return _rotate(x, positions, freqs, flags, mscale, x.new_empty(x.shape))

    @staticmethod
    def backward(ctx, g):
        positions, freqs = ctx.saved_tensors
        flags, mscale = ctx.how
        return _turn(g, positions, freqs, flags ^ B.HHR_ROPE_TRANSPOSE, mscale), None, None, None, None

    @staticmethod
    def jvp(ctx, tangent, *_):
        return _turn(tangent, *ctx.saved_tensors, *ctx.how)


def rope(x, positions, freqs, *, interleaved=False, mscale=1.0, out=None):
    """x [T, H, d] (bf16, fp16 or fp32; any token and head strides) with its first 2 * freqs.numel() elements
    rotated by positions[t] * freqs (hhr_rope).  positions: int32 [T]; freqs: float64 [rot/2].  Differentiable
    with respect to x, backward and forward (dual tensors).  out: where to put the result (x itself rotates in
    place; no other overlap with x); not with a gradient.  Captured into a CUDA graph, a backward pass wants leaves
    that no live eager graph holds: torch orders it behind that graph's stream."""
    shape = x.shape
    if len(shape) != 3 or x.dtype not in _TYPES or not x.is_cuda:
        raise ValueError(f"x: expected a bf16, fp16 or fp32 CUDA tensor [T, H, d], got {x.dtype} {tuple(x.shape)} on {x.device}")
    index = x.get_device()
    check_vector("positions", positions, torch.int32, shape[0], index)
    check_vector("freqs", freqs, torch.float64, freqs.numel(), index)
    flags, mscale = B.HHR_ROPE_INTERLEAVED if interleaved else 0, float(mscale)   # (the gradient takes this value, too)
    if (x.requires_grad or forward_ad._current_level >= 0) and _followed(x):
        if out is not None:
            raise ValueError("out= has no gradient: call without it, or on x.detach()")
        return _Rope.apply(x, positions, freqs, flags, mscale)
    if out is None:
        out = x.new_empty(shape)
    elif out.shape != shape or out.dtype is not x.dtype or out.get_device() != index or \
            (out.stride(2) != 1 and shape[2] > 1):
        raise ValueError(f"out: expected {x.dtype} {tuple(x.shape)} on {x.device} with adjacent elements of a head, "
                         f"got {out.dtype} {tuple(out.shape)} on {out.device}")
    elif out.requires_grad and torch.is_grad_enabled():
        raise ValueError("out= has no gradient: give it a tensor that needs none")
    else:
        written((out,))
    return _rotate(x, positions, freqs, flags, mscale, out)
