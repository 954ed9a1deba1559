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


TYPES = [(BF, BF), (FP16, FP16), (BF, E4), (FP16, E4)]


@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("n", [1, 3, 40, 2000])
def test_equal_logits_of_any_size_average_the_values(dtype, kv, n):
    """Keys that all give one logit x, up to what float32 holds: weights of 1 / n, and ln n + x.  The logits are powers
    of two, exact in every step, so the output has the errors of its float32 sums alone (n / 16 + 64 additions)."""
    c, q, t = make(1, 4, 2, 64, 16, 125, dtype=dtype, kv=kv)
    q.zero_()
    q[..., 5] = 16.0
    c.K.zero_()
    v = c.V.float()[t[0].long()].transpose(1, 2).reshape(2000, 2, 64)[:n].double().cpu()
    tol = 2.0 ** -24 * (n / 16 + 64) * v.abs().mean(0).repeat_interleave(2, 0)[None]
    for power in [0, 20, 23, 24, 25, 26, 27, 28, 30, 60, 100, 127]:
        for sign in (1.0, -1.0):
            c.K[..., 5] = torch.tensor(sign * 16.0).to(kv)
            x = sign * 2.0 ** power
            for out_dtype in (F32, dtype):
                out, lse, _ = attend(c, q, t, [n], out_dtype, scale=2.0 ** (power - 8))
                close(out, v.mean(0).repeat_interleave(2, 0)[None], tol)
                err = (lse.double().cpu() - (x + math.log(n))).abs().max()
                assert float(err) <= 2.0 ** -22 * abs(x + math.log(n)) + 2.0 ** -20, (power, sign)


@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("power", [23, 24, 25, 26])
def test_far_lower_logits_before_ordinary_ones(dtype, kv, power):
    """Whole tiles whose logits are -2^power, as a mask in the keys gives them, before and between ordinary tokens."""
    scales = (2.0 ** 6, 1.0) if kv == E4 else (1.0, 1.0)
    c, q, t = make(1, 4, 1, 128, 16, 60, dtype=dtype, kv=kv, scales=scales, hot=False)
    at = torch.arange(960)
    low = (at < 100) | ((at >= 300) & (at < 500)) | (at % 7 == 3) | (at > 900)
    n = torch.nonzero(low)[:, 0]
    q[..., 0] = 2.0 ** (power + 3 - 14)
    c.K[..., 0] = 0
    c.K[t[0].cpu()[n // 16].long().cuda(), 0, (n % 16).cuda(), 0] = torch.tensor(-2.0 ** 14 / scales[0]).to(kv)
    for out_dtype in (F32, dtype):
        out, lse, lens = attend(c, q, t, [960], out_dtype, scale=0.125)
        o, l, tol, ltol, _ = attend64(c, q, t, lens, scale=0.125, scales=scales, live=[~low])
        close(out, o, tol)
        assert bool(((lse.double().cpu() - l).abs() <= ltol).all())


@pytest.mark.parametrize("scale", [1.0, 0.5, 2.0])
def test_lowest_values_at_any_scale(scale):
    """A mask by the lowest bf16 value whose logit in powers of two (times log2 e) is beyond float32: alone it averages,
    before ordinary tokens it leaves no trace."""
    c, q, t = make(1, 4, 1, 64, 16, 8, hot=False)
    q[..., 0] = 1.0
    c.K[..., 0] = torch.finfo(BF).min
    out, _, _ = attend(c, q, t, [100], F32, scale=scale)
    v = c.V.float()[t[0].long()].transpose(1, 2).reshape(128, 64)[:100].double().cpu()
    if scale <= 1.0:      # (twice the lowest value is a logit of -inf)
        # the other products are below half a step of the mask's
        close(out, v.mean(0).expand(1, 4, 64), 2.0 ** -24 * 128 * v.abs().mean(0).expand(1, 4, 64))
    c.K[int(t[0, 5]), 0, 3:9, 0] = 0.0
    live = torch.zeros(128, dtype=torch.bool)
    live[83:89] = True
    out, lse, lens = attend(c, q, t, [100], F32, scale=scale)
    o, l, tol, ltol, _ = attend64(c, q, t, lens, scale=scale, live=[live])
    close(out, o, tol)
    assert bool(((lse.double().cpu() - l).abs() <= ltol).all())


# ---------------------------------------------------------------- float32 outputs

def bits16(w, dtype, terms):
    """w as a sum of 16-bit terms, each rounding what those before it leave."""
    out = torch.zeros_like(w)
    for _ in range(terms):
        out = out + (w - out).to(dtype).double()
    return out


@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("n", [2, 3, 9])
def test_weights_of_float32_outputs(dtype, kv, n):
    """A few tokens of nearly equal weights: the output has the roundings of its weights and hardly any of sums.  With
    e the logits' error: 4 e (two weights, over and under the line); ex2 of each, 2^-22, and the fp16 lift's rounding,
    2^-21.5, twice: 2^-20; the terms' rest, 2^-22; three 16-bit products, each a sum that may lose 2^-22; the sum of the
    weights, its inverse and the last product, 2^-22.  In all 4 e + 2^-20 + 5 2^-22.  Weights of one term less are
    further off than that (of two or three tokens; in nine they average out)."""
    c, q, t = make(8, 16, 2, 128, 16, 1, dtype=dtype, kv=kv, scales=(0.25, 2.0 ** -6) if kv == E4 else (1.0, 1.0), hot=False)
    scales = (c.desc.k_scale, c.desc.v_scale)
    q = (q.float() / 512).to(dtype)
    out, _, lens = attend(c, q, t, [n] * 8, F32)
    # the definition and, as a planted mistake, the same with coarser weights
    k = c.K.float()[t[:, 0].long()].double().cpu()[:, :, :n] * scales[0]
    v = c.V.float()[t[:, 0].long()].double().cpu()[:, :, :n] * scales[1]
    qd = q.double().cpu().view(8, 2, 8, 128)
    x = torch.einsum("bghd,bgnd->bghn", qd, k) / math.sqrt(128)
    e = (torch.einsum("bghd,bgnd->bghn", qd.abs(), k.abs()) / math.sqrt(128)).amax(-1, keepdim=True) * 132 * 2.0 ** -24
    w = torch.exp(x - x.amax(-1, keepdim=True))
    mix = lambda a: torch.einsum("bghn,bgnd->bghd", a, v) / w.sum(-1, keepdim=True)  # noqa: E731
    o = mix(w)
    tol = (4 * e + 2.0 ** -20 + 5 * 2.0 ** -22) * torch.einsum("bghn,bgnd->bghd", w, v.abs()) / w.sum(-1, keepdim=True)
    close(out, o.reshape(8, 16, 128), tol.reshape(8, 16, 128))
    products = BF if kv == BF else FP16
    if n > 3:
        return
    coarse = mix(bits16(w, products, 2 if products == BF else 1))
    assert int(((coarse - o).abs() > tol + 2.0 ** -24 * o.abs()).sum()) > 100


def long_units(dtype, n, out_dtype):
    """(out, its 64-bit value, tolerance without the output's rounding) of units that are one warp's each, n tokens long, all
    over the same pages; values are positive, so that an error in one direction adds up.

    Heads of 64 go in tiles of 32 tokens: n / 32 float32 additions of a tile's product to the output, n / 16 to a lane's sum
    of the weights, each off by 2^-24 of what has been summed so far, on average half of the end: 2^-24 (n / 64 + n / 32)
    on top of 4 e + 2^-20 + 5 2^-22 as above."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hkv, d = 8, 64
    B = -(-12 * min(sms, 160) // Hkv)
    g = torch.Generator().manual_seed(3)
    K = (torch.randn(n // 16, Hkv, 16, d, generator=g) / 8).to(dtype).cuda()
    V = (torch.rand(n // 16, Hkv, 16, d, generator=g) + 0.5).to(dtype).cuda()
    c = hhr.HHRPagedCache(q_heads=Hkv, kv_heads=Hkv, page=16, head_dim=d, dtype=dtype, K=K, V=V)
    q = (torch.randn(B, Hkv, d, generator=g) / 8).to(dtype).cuda()
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    out, _, _ = attend(c, q, table, [n] * B, out_dtype)
    k, v = (p.double().transpose(1, 2).reshape(n, Hkv, d) for p in (K, V))
    x = torch.einsum("bhd,nhd->bhn", q.double(), k) / 8
    e = (torch.einsum("bhd,nhd->bhn", q.double().abs(), k.abs()) / 8).amax(-1)[..., None] * 68 * 2.0 ** -24
    o = torch.einsum("bhn,nhd->bhd", torch.softmax(x, -1), v)
    tol = (4 * e + 2.0 ** -20 + 5 * 2.0 ** -22 + 2.0 ** -24 * (n / 64 + n / 32)) * o
    return out, o.cpu(), tol.cpu()


@pytest.mark.parametrize("dtype", [BF, FP16])
def test_sums_of_float32_outputs(dtype):
    """Sums that stay in the tensor cores from tile to tile lose about 1500 to 1900 2^-24 here, in one direction; the
    tolerance is about 800."""
    close(*long_units(dtype, 16384, F32))


@pytest.mark.parametrize("dtype", [BF, FP16])
def test_sums_of_16_bit_outputs(dtype):
    """Beside half a step of its type an output may be off by its float32 sums' tolerance, 1.9e-4 here.  Sums in the tensor
    cores lose 2.9e-4, more than half a step of fp16."""
    close(*long_units(dtype, 65536, dtype))
