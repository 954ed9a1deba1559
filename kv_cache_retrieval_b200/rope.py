"""Rotary positions on torch tensors: frequencies and the differentiable rotation."""
from __future__ import annotations

import torch

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


def on_device(device, fn, *args):
    """fn(*args, stream) with `device` current and torch's current stream of it."""
    if device.type != "cuda":
        raise ValueError(f"the buffers are on {device}: the library's kernels need a CUDA device")
    index = device.index
    if index == torch.cuda.current_device():
        return fn(*args, torch.cuda.current_stream(index).cuda_stream)
    with torch.cuda.device(index):
        return fn(*args, torch.cuda.current_stream(index).cuda_stream)


def check_tensor(name, t, dtype, device, shape=None):
    if t.dtype != dtype or t.device != device or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape) if shape is not None else ''} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _rotate(x, positions, freqs, interleaved, mscale, transpose, out):
    T, H, d = x.shape
    rot = B.hhr_rotation(2 * freqs.numel(), (B.HHR_ROPE_INTERLEAVED if interleaved else 0) |
                         (B.HHR_ROPE_TRANSPOSE if transpose else 0), mscale)
    if x.stride(2) != 1 and d > 1:
        x = x.contiguous()
    on_device(x.device, B.hhr_rope, T, H, d, _TYPES[x.dtype], rot, freqs, positions, x, x.stride(0), x.stride(1),
              out, out.stride(0), out.stride(1))
    return out


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions, freqs, interleaved, mscale):
        ctx.save_for_backward(positions, freqs)
        ctx.interleaved, ctx.mscale = interleaved, mscale
        return _rotate(x, positions, freqs, interleaved, mscale, False,
                       torch.empty(x.shape, dtype=x.dtype, device=x.device))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        # the Jacobian of a rotation is the rotation: its transpose gives the gradient
        positions, freqs = ctx.saved_tensors
        return _rotate(g, positions, freqs, ctx.interleaved, ctx.mscale, True,
                       torch.empty(g.shape, dtype=g.dtype, device=g.device)), None, None, None, None


def rope(x, positions, freqs, *, interleaved=False, mscale=1.0, out=None):
    """x [T, H, d] (bf16, fp16 or fp32; any token and head strides) with its first 2 * freqs.numel() elements
    rotated by positions[t] * freqs (hhr_rope).  positions: int32 [T]; freqs: float64 [rot/2].  Differentiable
    with respect to x.  out: where to put the result (x itself rotates in place); not with a gradient."""
    if x.dim() != 3 or x.dtype not in _TYPES or not x.is_cuda:
        raise ValueError(f"x: expected a bf16, fp16 or fp32 CUDA tensor [T, H, d], got {x.dtype} {tuple(x.shape)} on {x.device}")
    check_tensor("positions", positions, torch.int32, x.device, (x.shape[0],))
    check_tensor("freqs", freqs, torch.float64, x.device, (freqs.numel(),))
    if not positions.is_contiguous() or not freqs.is_contiguous():
        raise ValueError("positions and freqs have to be contiguous")
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out= has no gradient: call without it, or on x.detach()")
        return _Rope.apply(x, positions, freqs, interleaved, mscale)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        check_tensor("out", out, x.dtype, x.device, x.shape)
        if out.stride(2) != 1 and x.shape[2] > 1:
            raise ValueError("out: the elements of a head have to be adjacent")
    return _rotate(x, positions, freqs, interleaved, mscale, False, out)
