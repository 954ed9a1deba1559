"""The paged attention's arithmetic, tighter than tests/test_paged.py has it: every rounding on the way to an output is
counted, so that a term of the weights or a sum in fewer bits shows.

Let W = sum_n w_n |v_n| with the softmax weights w_n, and e the float32 error of the logits (attend64 there).  ex2.approx
is within 2^-22; it stands in the sum of the weights and in the products, so weights are off by 2^-21 + 2 e in all.
They are split into two 16-bit terms with at most 2^-17 (bf16) or 2^-22 (fp16) left over, or three of bf16 with 2^-25."""
import math

import pytest
import torch

import kv_cache_retrieval_b200 as hhr
from test_paged import BF, E4, F32, FP16, attend64, built, make  # noqa: F401 - built is a fixture
from test_rope import HALF

pytestmark = pytest.mark.gpu


def attend(c, q, t, lens, out_dtype, **kw):
    lens = torch.as_tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), dtype=F32, device="cuda")
    c.attend(q, t, lens, out=out, lse=lse, **kw)
    assert c.status() == hhr.HHR_OK
    return out, lse, lens


def close(out, o, tol):
    """out within tol of o and one rounding to its type: half a step at the size that the value may have."""
    top = (o.abs() + tol).clamp(min=2.0 ** -14 if out.dtype == FP16 else 2.0 ** -126)
    limit = tol + HALF[out.dtype] * torch.exp2(torch.floor(torch.log2(top)))
    err = (out.double().cpu() - o).abs()
    assert bool((err <= limit).all()), f"off by {float((err / limit).max())} of the tolerance, {int((err > limit).sum())} values"


@pytest.mark.parametrize("dtype", [BF, FP16])
@pytest.mark.parametrize("r", [4, 16])
def test_weights_of_an_8_bit_cache_are_not_rounded_to_16_bits(dtype, r):
    """A bf16 output rounds by 2^-8 at most, its weights by 2^-15 with everything else: a weight of one 16-bit term
    (2^-11) moves outputs that lie near the middle between two values further than that."""
    scales = (2.0 ** -5, 2.0 ** -6)
    c, q, t = make(4, 2 * r, 2, 128, 16, 40, dtype=dtype, kv=E4, scales=scales, hot=False)
    q = q / 16      # small logits: their own float32 error stays below the other roundings
    out, _, lens = attend(c, q, t, [640, 9, 100, 333], dtype)
    o, _, tol, _, _ = attend64(c, q, t, lens, scales=scales)
    close(out, o, tol)
