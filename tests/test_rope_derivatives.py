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


def test_a_saved_tensor_that_is_overwritten_is_noticed():
    """Writes in place and into out= raise the tensor's version: a graph that saved it refuses its backward pass."""
    f = _freqs(64)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    w = torch.ones((), device="cuda", requires_grad=True)
    x, room = _x((4, 2, 64), torch.float32), _x((4, 2, 64), torch.float32)
    for write in (lambda: hhr.rope(x, pos, f, out=x), lambda: hhr.rope(x, pos, f, out=room)):
        loss = (w * x * room).sum()
        write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    loss = (w * x).sum()
    hhr.rope(x, pos, f)
    loss.backward()
    with pytest.raises(ValueError):
        hhr.rope(x, pos, f, out=room.requires_grad_())
    with torch.no_grad():
        hhr.rope(x, pos, f, out=room)
    with torch.inference_mode():
        hhr.rope(x, pos, f, out=torch.empty_like(x))


def test_the_paged_calls_raise_the_versions_of_what_they_write():
    c = hhr.HHRPagedCache(q_heads=4, kv_heads=2, pages=4, page=16, head_dim=64)
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    q, out = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 4, 64, device="cuda")
    lse, table = torch.empty(1, 4, device="cuda"), torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    pos, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")

    def raised(call, *tensors):
        before = [t._version for t in tensors]
        call()
        return [t._version > b for t, b in zip(tensors, before)]

    assert raised(lambda: c.append(k, k, pos, table), c.K, c.V, k) == [True, True, False]
    assert raised(lambda: c.append(k, k, pos, table, q=q, q_out=q), c.K, c.V, q) == [True] * 3
    assert raised(lambda: c.attend(q, table, lens, out=out, lse=lse), out, lse, q, c.K) == [True, True, False, False]
    with torch.inference_mode():      # tensors without a version
        hhr.HHRPagedCache(q_heads=4, kv_heads=2, pages=4, page=16, head_dim=64).append(k, k, pos, table, q=q, q_out=q.clone())
