"""The rotation's derivatives beyond a backward pass: tangents of dual tensors, mixed orders, and writes that autograd has
to know of.  Tolerances as in test_rope.py."""
import pytest
import torch
from torch.autograd import forward_ad

import kv_cache_retrieval_b200 as hhr
from test_rope import _freqs, _x, built, check  # noqa: F401 - built is a fixture

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_the_tangent_is_rotated(dtype, interleaved):
    x, dx, f = _x((9, 3, 64), dtype), _x((9, 3, 64), dtype, 1), _freqs(48)
    pos = torch.arange(100, 109, dtype=torch.int32, device="cuda")
    with forward_ad.dual_level():
        y, dy = forward_ad.unpack_dual(hhr.rope(forward_ad.make_dual(x, dx), pos, f, interleaved=interleaved, mscale=1.25))
        assert forward_ad.unpack_dual(hhr.rope(x, pos, f)).tangent is None
        with pytest.raises(ValueError):
            hhr.rope(forward_ad.make_dual(x, dx), pos, f, out=torch.empty_like(x))
    check(y, x, pos, f, interleaved=interleaved, mscale=1.25)
    check(dy, dx, pos, f, interleaved=interleaved, mscale=1.25)


def test_the_tangent_of_a_gradient_and_the_gradient_of_a_tangent():
    x, dx, f = _x((5, 2, 64), torch.float32), _x((5, 2, 64), torch.float32, 1), _freqs(64)
    g, dg = _x((5, 2, 64), torch.float32, 2), _x((5, 2, 64), torch.float32, 3)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    leaf = x.clone().requires_grad_()
    with forward_ad.dual_level():      # forward over reverse: the gradient of an incoming dual one
        y = hhr.rope(leaf, pos, f)
        (gx,) = torch.autograd.grad(y, leaf, forward_ad.make_dual(g, dg))
        gx, dgx = forward_ad.unpack_dual(gx)
    check(gx, g, pos, f, transpose=True)
    check(dgx, dg, pos, f, transpose=True)
    tangent = dx.clone().requires_grad_()
    with forward_ad.dual_level():      # reverse over forward: the tangent's own gradient
        dy = forward_ad.unpack_dual(hhr.rope(forward_ad.make_dual(x, tangent), pos, f)).tangent
    (back,) = torch.autograd.grad(dy, tangent, g)
    check(back, g, pos, f, transpose=True)
