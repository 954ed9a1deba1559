"""The paged cache: appending tokens with their rotary positions, and the attention of one new token per sequence,
against 64 bits; what the calls refuse; bad pages and lengths; runs of the calls together.

Tolerances.  An appended element is the rotated one's float32 value (12 half steps of float32 on m (|x1| + |x2|), as in
test_rope.py) rounded once to the cache's type.  For attention let w_n be the softmax weights: the logits' float32
error is at most (d + 4) 2^-24 scale sum_e |q_e k_e| =: e_n for a d-term sum in any order and its scaling, which moves
each weight by a factor exp(+-2 max_n e_n); weights, sums and merges round to float32 (or a pair of 16-bit values that
holds 2^-16; with a bf16 output of an 8-bit cache one fp16 value, 2^-11), so with c = 2^-15 (or 2^-11 + 2^-15) + 2 max e_n
the output is within (c + 2^-24 rounds) sum_n w_n |v_n| + its own rounding.
The growth of float32 sums over n tokens is covered by 2^-24 (tokens of one lane + merges) <= 2^-24 (n / 16 + 64).  The
log-sum-exp is within max e_n + 2^-24 (n / 16 + 64) + 2^-22 |lse|."""
import ctypes as C
import math

import pytest
import torch

import kv_cache_retrieval_b200 as hhr
from kv_cache_retrieval_b200 import build as kbuild
from test_rope import HALF, exact

FAKE = 1 << 20
BF, FP16, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


# ---------------------------------------------------------------- refusals (host)

def desc(**kw):
    a = dict(Hq=8, Hkv=2, d=64, page=16, n_pages=10, table_cols=4, table_stride=4, q_type=0, kv_type=0, k_scale=1.0,
             v_scale=1.0, reserved=0, k_page=2048, k_head=1024, k_tok=64, v_page=2048, v_head=1024, v_tok=64)
    a.update(kw)
    return hhr.hhr_paged(*a.values())


BAD_DESC = [
    (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=7), 1), (dict(d=0), 1), (dict(d=96), 2), (dict(d=512), 2), (dict(page=0), 1),
    (dict(n_pages=0), 1), (dict(table_cols=0), 1), (dict(table_stride=3), 1), (dict(q_type=2), 1), (dict(q_type=3), 1),
    (dict(kv_type=1), 1), (dict(kv_type=2), 1), (dict(k_scale=2.0), 1), (dict(v_scale=0.5), 1), (dict(reserved=1), 1),
    (dict(kv_type=3, k_scale=0.0), 1), (dict(kv_type=3, v_scale=float("nan")), 1), (dict(kv_type=3, k_scale=-1.0), 1),
    (dict(kv_type=3, v_scale=float("inf")), 1), (dict(k_tok=60), 1), (dict(v_head=0), 1), (dict(k_page=-8), 1),
    (dict(kv_type=3, k_tok=72), 1), (dict(page=1 << 20, table_cols=1 << 11, table_stride=1 << 11), 2)]


def attend(c, B=3, q=FAKE, q_seq=512, K=FAKE, V=FAKE, table=FAKE, lens=FAKE, window=0, scale=0.1, out_type=0, out=FAKE,
           lse=None, ws=FAKE, ws_bytes=1 << 30):
    return hhr.lib().hhr_paged_attend(C.byref(c), B, q, q_seq, K, V, table, lens, window, scale, out_type, out, lse, ws,
                                      ws_bytes, None)


def append(c, T=3, B=3, rotation="default", freqs=FAKE, pos=FAKE, rope_pos=None, seq=None, table=FAKE, q=None, q_tok=512,
           q_out=None, q_out_tok=512, k=FAKE, k_row=128, v=FAKE, v_row=128, K=FAKE, V=FAKE, status=None, rot=64, flags=0):
    r = None if rotation is None else C.byref(hhr.hhr_rotation(rot, flags, 1.0))
    return hhr.lib().hhr_paged_append(C.byref(c), T, B, r, freqs, pos, rope_pos, seq, table, q, q_tok, q_out, q_out_tok, k,
                                      k_row, v, v_row, K, V, status, None)


@pytest.mark.parametrize("kw,status", BAD_DESC)
def test_bad_descriptions(kw, status):
    assert attend(desc(**kw)) == status
    assert append(desc(**kw)) == status
    assert hhr.hhr_paged_workspace_size(desc(**kw)) == 0


def test_workspace_size():
    assert hhr.hhr_paged_workspace_size(desc()) > 0
    assert hhr.hhr_paged_workspace_size(desc()) % 256 == 0
    # it follows the cache, not the pool or the table
    assert hhr.hhr_paged_workspace_size(desc()) == hhr.hhr_paged_workspace_size(desc(n_pages=1 << 20, table_cols=1 << 15,
                                                                                    table_stride=1 << 15))


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(window=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(out_type=1), 1),
    (dict(out_type=3), 1), (dict(q=None), 1), (dict(K=None), 1), (dict(V=None), 1), (dict(table=None), 1),
    (dict(lens=None), 1), (dict(out=None), 1), (dict(q=FAKE + 8), 1), (dict(K=FAKE + 8), 1), (dict(out=FAKE + 2), 1),
    (dict(lens=FAKE + 2), 1), (dict(lse=FAKE + 2), 1), (dict(q_seq=-8), 1), (dict(q_seq=516), 1), (dict(ws=None), 3),
    (dict(ws=FAKE + 16), 3), (dict(ws_bytes=128), 3), (dict(B=1 << 29), 2)])
def test_attend_refusals(kw, status):
    assert attend(desc(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(B=-1), 1), (dict(T=4), 1), (dict(q=FAKE), 1), (dict(q_out=FAKE), 1), (dict(rot=66), 1),
    (dict(rot=7), 1), (dict(flags=2), 1), (dict(flags=8), 1), (dict(freqs=None), 1), (dict(k_row=-1), 1),
    (dict(v_row=-1), 1), (dict(q=FAKE, q_out=FAKE * 2, q_tok=-1), 1), (dict(q=FAKE, q_out=FAKE * 2, q_out_tok=511), 1),
    (dict(q=FAKE, q_out=FAKE, q_tok=1024), 1), (dict(pos=None), 1), (dict(table=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(K=None), 1), (dict(V=None), 1), (dict(K=FAKE + 8), 1), (dict(pos=FAKE + 1), 1),
    (dict(seq=FAKE + 2), 1), (dict(rope_pos=FAKE + 2), 1), (dict(status=FAKE + 2), 1), (dict(k=FAKE + 1), 1),
    (dict(T=1 << 30, B=1 << 30), 2)])
def test_append_refusals(kw, status):
    assert append(desc(), **kw) == status


def test_nothing_to_do_is_ok():
    assert attend(desc(), B=0, q=None, lens=None) == hhr.HHR_OK
    assert append(desc(), T=0, pos=None, k=None) == hhr.HHR_OK
    assert hhr.lib().hhr_paged_attend(None, 1, FAKE, 0, FAKE, FAKE, FAKE, FAKE, 0, 0.1, 0, FAKE, None, FAKE, 1 << 30,
                                      None) == hhr.HHR_ERR_INVALID_ARG


def test_status_string_of_a_bad_index():
    assert hhr.hhr_status_string(hhr.HHR_ERR_BAD_INDEX) not in ("ok", "unknown status")


def test_cache_object_refusals():
    base = dict(q_heads=8, kv_heads=2, pages=4, head_dim=64, device="cpu")
    for bad in (dict(layout="rows"), dict(dtype=F32), dict(kv_dtype=FP16), dict(pages=None), dict(K=torch.zeros(4, 2, 16, 64))):
        with pytest.raises(ValueError):
            hhr.HHRPagedCache(**{**base, **bad})
    for bad in (dict(head_dim=96), dict(kv_heads=3), dict(k_scale=2.0), dict(kv_dtype=E4, k_scale=0.0)):
        with pytest.raises(hhr.HhrError):
            hhr.HHRPagedCache(**{**base, **bad})
    K = torch.zeros(4, 2, 16, 64, dtype=BF)
    for k, v in ((K, K.half()), (K[:3], K), (K, torch.zeros(4, 2, 64, 16, dtype=BF).transpose(2, 3))):
        with pytest.raises(ValueError):
            hhr.HHRPagedCache(**{**base, "K": k, "V": v})
    c = hhr.HHRPagedCache(**base)
    t = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):     # buffers that are not on a CUDA device
        c.attend(torch.zeros(1, 8, 64, dtype=BF), t, torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        c.append(torch.zeros(1, 2, 64, dtype=BF), torch.zeros(1, 2, 64, dtype=BF), torch.zeros(1, dtype=torch.int32), t)


# ---------------------------------------------------------------- the definitions in 64 bits (CPU)

def as64(pool):
    return pool.float().double().cpu()


def tokens(cache, pool, table, b, lo, n):
    """[tokens, Hkv, d] in float64 of tokens lo .. n of sequence b."""
    page = cache.desc.page
    at = torch.arange(lo, n)
    ids, off = table.cpu()[b].long()[at // page], at % page
    x = as64(pool)
    return x[ids, :, off] if cache.head_major else x[ids, off]


def attend64(cache, q, table, lens, window=0, scale=None, scales=(1.0, 1.0), live=None):
    """out, lse and their tolerances (without the output type's rounding) in float64; live[b]: a mask of the tokens."""
    B, Hq, d = q.shape
    Hkv = cache.desc.Hkv
    r = Hq // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    q = q.double().cpu()
    out, tol = torch.zeros(B, Hq, d, dtype=torch.float64), torch.zeros(B, Hq, d, dtype=torch.float64)
    mag = torch.zeros(B, Hq, d, dtype=torch.float64)
    lse, ltol = torch.full((B, Hq), -math.inf, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    for b, n in enumerate(lens.tolist()):
        lo = max(0, n - window) if window else 0
        if n <= lo:
            continue
        k, v = (tokens(cache, p, table, b, lo, n) * s for p, s in zip((cache.K, cache.V), scales))
        if live is not None:
            k, v = k[live[b][lo:n]], v[live[b][lo:n]]
            if k.shape[0] == 0:
                continue
        for h in range(Hq):
            x = k[:, h // r] @ q[b, h] * scale
            e = ((k[:, h // r].abs() @ q[b, h].abs()) * abs(scale)).max() * (d + 4) * 2.0 ** -24
            lse[b, h] = torch.logsumexp(x, 0)
            w = torch.exp(x - lse[b, h])
            out[b, h] = w @ v[:, h // r]
            sums = 2.0 ** -24 * (k.shape[0] / 16 + 64)
            mag[b, h] = w @ v[:, h // r].abs()
            tol[b, h] = (2.0 ** -15 + 2 * e + sums) * mag[b, h]
            ltol[b, h] = e + sums + 2.0 ** -22 * lse[b, h].abs()
    return out, lse, tol, ltol, mag


def compare(out, lse, want, name="", rounded=0.0):
    """rounded: what the weights' own rounding adds, relative to sum w |v| (attend64 has 2^-15 of it)."""
    o, l, tol, ltol, mag = want
    tol = tol + rounded * mag
    half = HALF[out.dtype]
    err = (out.double().cpu() - o).abs()
    limit = half * o.abs() + tol * (1 + half) + (2.0 ** -25 if out.dtype == FP16 else 0.0)
    assert bool((err <= limit).all()), f"{name}: out off by {float((err / (limit + 1e-300)).max())} of the tolerance"
    if lse is not None:
        l64 = lse.double().cpu()
        assert torch.equal(torch.isinf(l64), torch.isinf(l)), f"{name}: empty rows differ"
        ok = ~torch.isinf(l)
        assert bool(((l64 - l).abs()[ok] <= ltol[ok]).all()), f"{name}: lse off"


def make(B, Hq, Hkv, d, page, cols, *, dtype=BF, kv=None, layout="head", seed=0, spare=3, scales=(1.0, 1.0), hot=True):
    """A cache whose pool is full of numbers and a table of distinct, shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    pages = B * cols + spare
    kv = kv or dtype
    c = hhr.HHRPagedCache(q_heads=Hq, kv_heads=Hkv, pages=pages, page=page, head_dim=d, dtype=dtype, kv_dtype=kv,
                          layout=layout, k_scale=scales[0], v_scale=scales[1])
    c.head_major = layout == "head"
    for p, s in ((c.K, scales[0]), (c.V, scales[1])):
        x = torch.randn(p.shape, generator=g) / s
        p.copy_(x.clamp(-448, 448).to(kv))
    q = torch.randn(B, Hq, d, generator=g) * (2.0 if hot else 1.0)
    table = torch.randperm(pages, generator=g)[:B * cols].view(B, cols).to(torch.int32).cuda()
    return c, q.to(dtype).cuda(), table


def run(c, q, table, lens, *, window=0, out_dtype=None, scales=(1.0, 1.0), name="", low=None, **kw):
    """low: tokens whose weight is zero by their logits' size (left out of the tolerance's largest logit)."""
    lens = torch.as_tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=out_dtype or q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), dtype=F32, device="cuda")
    got = c.attend(q, table, lens, out=out, lse=lse, window=window, **kw)
    assert got is out
    torch.cuda.synchronize()
    assert c.status() == hhr.HHR_OK
    compare(out, lse, attend64(c, q, table, lens, window, kw.get("scale"), scales, None if low is None else [~low]), name,
            2.0 ** -11 if c.K.dtype == E4 and out.dtype == BF else 0.0)
    return out, lse


# ---------------------------------------------------------------- attention

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", [(BF, BF), (FP16, FP16), (BF, E4), (FP16, E4)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("r", [1, 3, 4, 8, 9, 16, 24])
def test_attend_types_and_groups(dtype, kv, d, r):
    scales = (2.0 ** -5, 2.0 ** -6) if kv == E4 else (1.0, 1.0)
    c, q, t = make(3, 2 * r, 2, d, 16, 20, dtype=dtype, kv=kv, scales=scales)
    run(c, q, t, [300, 1, 77], out_dtype=F32, scales=scales)
    run(c, q, t, [16, 0, 320], scales=scales)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("page,cols", [(1, 200), (2, 70), (5, 41), (8, 30), (16, 17), (20, 11), (32, 9), (48, 5), (64, 4),
                                       (100, 3), (257, 1), (1000, 2)])
def test_attend_pages(page, cols, layout):
    c, q, t = make(4, 8, 2, 64, page, cols, layout=layout)
    cap = page * cols
    run(c, q, t, [cap, cap - 1, max(0, cap // 2 + 1), min(cap, 17)], out_dtype=F32)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 255, 256, 257, 1023, 2049, 4097])
def test_attend_lengths(n):
    c, q, t = make(1, 8, 2, 128, 16, 257)
    run(c, q, t, [n], out_dtype=F32)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 999, 5000])
def test_attend_window(window):
    c, q, t = make(5, 6, 2, 64, 16, 70)
    run(c, q, t, [1120, 1, 0, 517, 129], window=window, out_dtype=F32)


@pytest.mark.gpu
def test_attend_many_ragged_sequences():
    c, q, t = make(130, 8, 2, 64, 16, 12, layout="token")
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 193, (130,), generator=g)
    lens[::7] = 0
    lens[-1] = 0
    run(c, q, t, lens.tolist())


@pytest.mark.gpu
def test_attend_more_sequences_than_threads_of_a_block():
    c, q, t = make(1500, 4, 1, 64, 16, 2)
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 33, (1500,), generator=g)
    lens[:700] = 0
    run(c, q, t, lens.tolist())
    run(c, q, t, [0] * 1500)
    run(c, q, t, [0] * 1499 + [3])


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d", [(32, 1, 128), (71, 1, 64), (40, 1, 256), (128, 2, 128), (33, 33, 64), (100, 4, 128)])
def test_attend_head_counts(Hq, Hkv, d):
    c, q, t = make(2, Hq, Hkv, d, 16, 40)
    run(c, q, t, [640, 333], out_dtype=F32)


@pytest.mark.gpu
def test_attend_long_context_split_over_the_card():
    c, q, t = make(1, 8, 2, 128, 16, 2500, hot=False)
    run(c, q, t, [39999], out_dtype=F32)
    run(c, q, t, [39999])
    c, q, t = make(2, 4, 2, 128, 16, 2000, kv=E4, scales=(2.0 ** -5, 2.0 ** -5), hot=False)
    run(c, q, t, [31999, 5], out_dtype=F32, scales=(2.0 ** -5, 2.0 ** -5))


@pytest.mark.gpu
def test_attend_is_the_same_every_time():
    c, q, t = make(3, 8, 2, 128, 16, 600)
    lens = torch.tensor([9600, 4001, 17], dtype=torch.int32, device="cuda")
    first = c.attend(q, t, lens, out=torch.empty(q.shape, device="cuda"))
    for _ in range(20):
        assert torch.equal(c.attend(q, t, lens, out=torch.empty(q.shape, device="cuda")), first)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", [BF, E4])
def test_attend_does_not_read_beyond_a_sequence(kv):
    """NaN in every place that is not a token of the sequences: the rest of the last page, the places before the window,
    other pages; bad page numbers behind the last page."""
    scales = (0.25, 0.25) if kv == E4 else (1.0, 1.0)
    c, q, t = make(3, 8, 2, 64, 16, 10, kv=kv, scales=scales)
    lens, window = [150, 37, 0], 20
    K, V = c.K.clone(), c.V.clone()
    nan = torch.full((1,), float("nan"), device="cuda").to(kv)
    c.K.view(torch.uint8).copy_(nan.expand(c.K.shape).contiguous().view(torch.uint8).view(c.K.view(torch.uint8).shape))
    c.V.view(torch.uint8).copy_(c.K.view(torch.uint8))
    for b, n in enumerate(lens):
        for i in range(max(0, n - window), n):
            p = int(t[b, i // 16])
            for dst, src in ((c.K, K), (c.V, V)):
                dst.view(torch.uint8)[p, :, i % 16] = src.view(torch.uint8)[p, :, i % 16]
    t[1, 3:] = -5
    t[1, 0] = 1 << 30            # before the window
    t[2, :] = 1 << 29
    run(c, q, t, lens, window=window, scales=scales, out_dtype=F32)


@pytest.mark.gpu
def test_attend_extreme_values():
    c, q, t = make(1, 4, 1, 64, 16, 8)
    # a logit far above the others late in the sequence, and large negative ones
    c.K[int(t[0, 6]), 0, 3] = (q[0, 0] * 20).to(BF)
    c.K[int(t[0, 1]), 0, 5] = (q[0, 0] * -20).to(BF)
    run(c, q, t, [128], out_dtype=F32)
    # logits of -inf leave their tokens out; a row of nothing else is empty
    q2 = torch.zeros_like(q)
    q2[..., 0] = 1.0
    c.K[..., 0] = -math.inf
    out = torch.full(q.shape, 5.0, device="cuda")
    lse = torch.zeros(1, 4, device="cuda")
    c.attend(q2, t, torch.tensor([100], dtype=torch.int32, device="cuda"), out=out, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    c.K[int(t[0, 2]), 0, 1, 0] = 1.0
    c.attend(q2, t, torch.tensor([100], dtype=torch.int32, device="cuda"), out=out, lse=lse)
    v = c.V[int(t[0, 2]), 0, 1].float()
    assert torch.equal(out[0, 0], v) and float((lse - 0.125).abs().max()) <= 2.0 ** -20
    # the type's lowest value as a mask: its token has no weight beside any other
    c.K[..., 0] = torch.finfo(BF).min
    c.K[int(t[0, 2]), 0, 1, 0] = 1.0
    c.attend(q2, t, torch.tensor([100], dtype=torch.int32, device="cuda"), out=out, lse=lse)
    assert torch.equal(out[0, 0], v)
    # NaN in a key of a sequence reaches that sequence's outputs
    c.K[int(t[0, 2]), 0, 1, 0] = math.nan
    c.attend(q2, t, torch.tensor([100], dtype=torch.int32, device="cuda"), out=out, lse=lse)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_attend_lowest_values_beside_ordinary_ones(d):
    """Keys that give the type's lowest logits in whole tiles before, between and behind ordinary ones: the ordinary
    ones keep their differences."""
    c, q, t = make(1, 4, 1, d, 16, 60)
    q[..., 0] = 1.0
    at = torch.arange(960)
    low = (at < 100) | ((at >= 300) & (at < 500)) | (at % 7 == 3) | (at > 900)
    n = torch.nonzero(low)[:, 0]
    c.K[t[0].cpu()[n // 16].long().cuda(), 0, (n % 16).cuda(), 0] = torch.finfo(BF).min
    run(c, q, t, [960], out_dtype=F32, low=low)
    run(c, q, t, [95], out_dtype=F32, low=None)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-30, 3.0])
@pytest.mark.parametrize("kv", [BF, E4])
def test_attend_scales(scale, kv):
    scales = (2.0 ** -5, 2.0 ** -5) if kv == E4 else (1.0, 1.0)
    c, q, t = make(2, 6, 2, 64, 16, 20, kv=kv, scales=scales)
    run(c, q, t, [301, 7], out_dtype=F32, scale=scale, scales=scales)


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-60, 0, 60])
def test_attend_e4m3_with_queries_of_any_size(power):
    """bf16 queries have a far wider range than the 16-bit products of an 8-bit cache: their rows keep their size."""
    scales = (2.0 ** -5, 2.0 ** -5)
    c, q, t = make(2, 8, 2, 64, 16, 10, kv=E4, scales=scales)
    q = (q.float() * 2.0 ** power).to(BF)
    q[1, 3] = 0
    run(c, q, t, [160, 33], out_dtype=F32, scales=scales, scale=0.125 * 2.0 ** -power)


@pytest.mark.gpu
def test_attend_every_e4m3_value():
    """A cache holding each 8-bit pattern, NaN aside, once as a value and once as a key."""
    c, q, t = make(1, 2, 1, 64, 16, 16, kv=E4, scales=(2.0 ** -9, 1.0))
    codes = torch.arange(256, dtype=torch.uint8)
    codes[(codes & 0x7f) == 0x7f] = 0
    for i in range(256):
        p = int(t[0, i // 16])
        c.K.view(torch.uint8)[p, 0, i % 16] = codes.roll(i)[:64].cuda()
        c.V.view(torch.uint8)[p, 0, i % 16] = codes.roll(-i)[:64].cuda()
    run(c, q, t, [256], out_dtype=F32, scales=(2.0 ** -9, 1.0))


@pytest.mark.gpu
def test_attend_bad_indices_are_reported_and_masked():
    c, q, t = make(4, 8, 2, 64, 16, 6)
    lens = torch.tensor([96, 97, -1, 50], dtype=torch.int32, device="cuda")
    t[0, 2] = -1
    t[3, 3] = c.desc.n_pages
    out = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    c.attend(q, t, lens, out=out, lse=lse)
    assert c.status() == hhr.HHR_ERR_BAD_INDEX
    assert c.status() == hhr.HHR_OK
    live = [torch.ones(96, dtype=torch.bool) for _ in range(4)]
    live[0][32:48] = False
    live[3][48:64] = False
    safe = t.clone()
    safe[0, 2] = safe[3, 3] = 0
    want = attend64(c, q, safe, torch.tensor([96, 0, 0, 50]), live=live)
    compare(out, lse, want)
    run(c, q, safe, [96, 0, 1, 50])      # the workspace is as it was


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 5])
def test_attend_with_no_valid_page_at_all(page):
    c, q, t = make(2, 4, 2, 64, page, 8)
    t[1] = -1
    out = torch.full(q.shape, float("nan"), device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    c.attend(q, t, torch.tensor([8 * page] * 2, dtype=torch.int32, device="cuda"), out=out, lse=lse)
    assert c.status() == hhr.HHR_ERR_BAD_INDEX
    live = [torch.ones(8 * page, dtype=torch.bool), torch.zeros(8 * page, dtype=torch.bool)]
    compare(out, lse, attend64(c, q, t.clamp(min=0), torch.tensor([8 * page] * 2), live=live))
    assert bool((out[1] == 0).all())


@pytest.mark.gpu
def test_attend_strides_and_views():
    """A pool that is a view of a larger buffer with K and V interleaved, query rows inside the projection's, a table
    that is a slice, sequences that share pages, a page used twice."""
    g = torch.Generator().manual_seed(8)
    buf = torch.randn(30, 2, 16, 3, 64, generator=g).to(BF).cuda()      # [pages][K / V][page][heads + 1][d]
    K, V = buf[:, 0, :, :2], buf[:, 1, :, :2]
    c = hhr.HHRPagedCache(q_heads=8, kv_heads=2, page=16, head_dim=64, K=K, V=V, layout="token")
    c.head_major = False
    rows = torch.randn(3, 12, 64, generator=g).to(BF).cuda()
    wide = torch.randint(0, 30, (3, 9), generator=g, dtype=torch.int32).cuda()
    table = wide[:, 2:7]
    table[2] = table[0]
    table[1, 3] = table[1, 0]
    run(c, rows[:, 2:10], table, [80, 71, 80], out_dtype=F32)
    # heads of the pool before tokens, pages last but one
    buf = torch.randn(2, 30, 64 + 8, 64, generator=g).to(BF).cuda()
    K = buf[:, :, :16].transpose(0, 1)
    V = buf[:, :, 24:40].transpose(0, 1)
    c = hhr.HHRPagedCache(q_heads=8, kv_heads=2, page=16, head_dim=64, K=K, V=V)
    c.head_major = True
    run(c, rows[:, :8], table, [80, 71, 80], out_dtype=F32)


@pytest.mark.gpu
def test_attend_offsets_beyond_32_bits():
    """Pools of 9 GiB whose last pages lie past 2^32 elements."""
    d, Hkv, page = 128, 8, 64
    pages = (1 << 32) // (d * Hkv * page) + 40
    K = torch.empty(pages, Hkv, page, d, dtype=BF, device="cuda")
    V = torch.empty_like(K)
    for i, p in enumerate((K, V)):
        p[-40:] = torch.randn(40, Hkv, page, d, generator=torch.Generator().manual_seed(i)).to(BF).cuda()
    c = hhr.HHRPagedCache(q_heads=16, kv_heads=Hkv, page=page, head_dim=d, K=K, V=V)
    q = torch.randn(1, 16, d, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    last = torch.arange(pages - 40, pages, dtype=torch.int32, device="cuda").flip(0)
    small = hhr.HHRPagedCache(q_heads=16, kv_heads=Hkv, page=page, head_dim=d, K=K[-40:], V=V[-40:])
    n = torch.tensor([40 * page - 3], dtype=torch.int32, device="cuda")
    a = c.attend(q, last.view(1, 40), n)
    b = small.attend(q, (last - (pages - 40)).view(1, 40).contiguous(), n)
    assert torch.equal(a, b)
    # and the append's
    k, v = (torch.randn(1, Hkv, d, generator=torch.Generator().manual_seed(i)).to(BF).cuda() for i in (3, 4))
    c.append(k, v, torch.tensor([7], dtype=torch.int32, device="cuda"), last.view(1, 40))
    assert torch.equal(K[pages - 1, :, 7], k[0]) and torch.equal(V[pages - 1, :, 7], v[0])


@pytest.mark.gpu
def test_attend_checks():
    c, q, t = make(2, 8, 2, 64, 16, 6)
    lens = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    for bad in (dict(q=q[:1]), dict(q=q[:, :7]), dict(q=q.half()), dict(table=t.long()), dict(table=t[0]),
                dict(table=t.t()), dict(lens=lens.long()), dict(lens=lens[:1]), dict(lens=lens.cpu()),
                dict(out=torch.empty(2, 8, 64, dtype=FP16, device="cuda")), dict(out=torch.empty(2, 8, 32, dtype=BF, device="cuda")),
                dict(lse=torch.empty(2, 8, dtype=BF, device="cuda")), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(q=q, table=t, lens=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            c.attend(a.pop("q"), a.pop("table"), a.pop("lens"), **a)
    with pytest.raises(hhr.HhrError):
        c.attend(q, t, lens, window=-1)
    with pytest.raises(hhr.HhrError):
        c.attend(q, t, lens, scale=float("nan"))
    with pytest.raises(hhr.HhrError):
        c.attend(q, t, lens, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert c.attend(q[:0], t[:0], lens[:0]).shape == (0, 8, 64)


# ---------------------------------------------------------------- append

def near(got, want, mag, dtype, scale):
    """got (the stored type) against want (float64): one rounding of the float32 value."""
    slack = 12 * 2.0 ** -24 * mag / scale
    if dtype == E4:
        y = want / scale
        lo, hi = (y - slack), (y + slack)
        g = got.float().double().cpu()
        near_e4 = lambda z: z.clamp(-448, 448).float().to(E4).float().double()  # noqa: E731
        a, b = near_e4(lo), near_e4(hi)
        return bool(((g >= a) & (g <= b)).all())
    err = (got.double().cpu() - want).abs()
    return bool((err <= HALF[dtype] * want.abs() + slack * (1 + HALF[dtype]) + (2.0 ** -25 if dtype == FP16 else 0)).all())


def check_append(c, K0, V0, k, v, pos, table, seq=None, q=None, q_out=None, freqs=None, rope_pos=None, interleaved=False,
                 mscale=1.0, scales=(1.0, 1.0)):
    d = c.desc
    fz = torch.empty(0, dtype=torch.float64) if freqs is None else freqs
    turn = dict(mscale=mscale, interleaved=interleaved)
    ky, kmag = exact(k, pos if rope_pos is None else rope_pos, fz, **turn)
    untouched = torch.ones(c.K.shape[0], d.page, dtype=torch.bool)
    dtype = c.K.dtype
    view = (lambda x: x) if not c.head_major else (lambda x: x.transpose(1, 2))
    raw = (lambda x: x.view(torch.uint8)) if dtype == E4 else (lambda x: x.view(torch.int16))
    for t in range(k.shape[0]):
        p, s = int(pos[t]), t if seq is None else int(seq[t])
        if p < 0:
            continue
        id, off = int(table[s, p // d.page]), p % d.page
        untouched[id, off] = False
        assert near(view(c.K)[id, off], ky[t], kmag[t], dtype, scales[0]), f"key {t}"
        assert near(view(c.V)[id, off], v[t].double().cpu(), 0 * kmag[t], dtype, scales[1]), f"value {t}"
    same = untouched.cuda()
    for now, was in ((c.K, K0), (c.V, V0)):
        a, b = raw(view(now)), raw(view(was))
        assert bool((a == b)[same].all()), "a place that no token names changed"
    if q is not None:
        qy, qmag = exact(q, pos if rope_pos is None else rope_pos, fz, **turn)
        live = (pos >= 0).cpu()
        assert near(q_out[live.cuda()], qy[live], qmag[live], q.dtype, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kv", [(BF, BF), (FP16, FP16), (BF, E4), (FP16, E4)])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 32), (128, 128), (256, 64), (128, 90), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(dtype, kv, d, rot, interleaved):
    scales = (2.0 ** -4, 2.0 ** -6) if kv == E4 else (1.0, 1.0)
    c, _, t = make(5, 6, 2, d, 16, 6, dtype=dtype, kv=kv, scales=scales, layout="token" if interleaved else "head")
    g = torch.Generator().manual_seed(1)
    T = 43
    rows = torch.randn(T, 10, d, generator=g).to(dtype).cuda()
    q, k, v = rows.split([6, 2, 2], dim=1)
    at = torch.randperm(5 * 96, generator=g)[:T]
    seq, pos = (at // 96).to(torch.int32).cuda(), (at % 96).to(torch.int32).cuda()
    pos[7] = pos[20] = -1
    f = hhr.rope_freqs(rot)[0] if rot else None
    K0, V0 = c.K.clone(), c.V.clone()
    keep = torch.full((T, 6, d), 3.0, dtype=dtype, device="cuda")
    out = c.append(k, v, pos, t, seq=seq, q=q, q_out=keep, freqs=f, interleaved=interleaved, mscale=1.125 if rot else 1.0)
    assert out is keep and c.status() == hhr.HHR_OK
    check_append(c, K0, V0, k, v, pos, t, seq, q, out, f, interleaved=interleaved, mscale=1.125 if rot else 1.0, scales=scales)
    assert bool((keep[pos < 0] == 3.0).all())        # nothing of a padding row is written


@pytest.mark.gpu
@pytest.mark.parametrize("page,layout", [(1, "head"), (7, "token"), (16, "head"), (64, "token"), (1000, "head")])
def test_append_one_token_of_each_sequence(page, layout):
    cols = max(2, 128 // page)
    c, q, t = make(6, 8, 4, 128, page, cols, layout=layout)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(6, 4, 128, generator=g).to(BF).cuda() for _ in range(2))
    pos = torch.randint(0, page * cols, (6,), generator=g, dtype=torch.int32).cuda()
    f = hhr.rope_freqs(128, base=5e5, scaling="bands", factor=8.0, orig=8192)[0]
    K0, V0 = c.K.clone(), c.V.clone()
    far = pos + 100000
    out = c.append(k, v, pos, t, q=q, freqs=f, rope_positions=far)
    check_append(c, K0, V0, k, v, pos, t, None, q, out, f, rope_pos=far)
    # in place, and without queries
    K0, V0 = c.K.clone(), c.V.clone()
    q1 = q.clone()
    assert c.append(k, v, pos, t, q=q1, q_out=q1, freqs=f) is q1
    check_append(c, K0, V0, k, v, pos, t, None, q, q1, f)
    assert c.append(k, v, pos, t) is None
    check_append(c, K0, V0, k, v, pos, t)


@pytest.mark.gpu
def test_append_prompt_of_many_tokens():
    c, _, t = make(3, 8, 2, 64, 16, 70)
    g = torch.Generator().manual_seed(5)
    T = 2111
    q, k, v = (torch.randn(T, h, 64, generator=g).to(BF).cuda() for h in (8, 2, 2))
    seq = torch.cat([torch.full((n,), i) for i, n in enumerate((1000, 1, 1110))]).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(120, 1120), torch.tensor([77]), torch.arange(0, 1110)]).to(torch.int32).cuda()
    f = hhr.rope_freqs(64)[0]
    K0, V0 = c.K.clone(), c.V.clone()
    out = c.append(k, v, pos, t, seq=seq, q=q, freqs=f)
    check_append(c, K0, V0, k, v, pos, t, seq, q, out, f)


@pytest.mark.gpu
def test_append_odd_strides_and_alignment():
    """Rows that no 16-byte access can take: odd token strides and an odd first element."""
    c, _, t = make(2, 4, 2, 64, 16, 4)
    g = torch.Generator().manual_seed(6)
    flat = torch.randn(9 * 601 + 1, generator=g).to(BF).cuda()
    rows = flat[1:].as_strided((9, 8, 64), (601, 64, 1))
    q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:]
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    seq = torch.ones(9, dtype=torch.int32, device="cuda")
    room = torch.zeros(9 * 333, dtype=BF, device="cuda").as_strided((9, 4, 64), (333, 64, 1))
    f = hhr.rope_freqs(64)[0]
    K0, V0 = c.K.clone(), c.V.clone()
    c.append(k, v, pos, t, seq=seq, q=q, q_out=room, freqs=f)
    check_append(c, K0, V0, k, v, pos, t, seq, q, room, f)


@pytest.mark.gpu
def test_append_e4m3_saturates_and_keeps_nan():
    c, _, t = make(1, 2, 1, 64, 16, 1, kv=E4, scales=(0.5, 0.25))
    k, v = (torch.zeros(1, 1, 64, dtype=BF, device="cuda") for _ in range(2))
    k[0, 0, :6] = torch.tensor([1e6, -1e6, 224.0, 232.0, 0.0, -0.0])
    k[0, 0, 6], v[0, 0, 0], v[0, 0, 1], v[0, 0, 2] = math.nan, math.inf, -math.inf, 2.0 ** -12
    c.append(k, v, torch.tensor([3], dtype=torch.int32, device="cuda"), t)
    p = int(t[0, 0])
    got = c.K[p, 0, 3].float().cpu()
    assert got[:4].tolist() == [448.0, -448.0, 448.0, 448.0] and bool(torch.isnan(got[6])) and bool((got[7:] == 0).all())
    assert c.V[p, 0, 3].float().cpu()[:3].tolist() == [448.0, -448.0, 2.0 ** -9 * 0.0]


@pytest.mark.gpu
def test_append_bad_indices():
    c, q, t = make(3, 4, 2, 64, 16, 4)
    g = torch.Generator().manual_seed(9)
    T = 7
    k, v = (torch.randn(T, 2, 64, generator=g).to(BF).cuda() for _ in range(2))
    qt = torch.randn(T, 4, 64, generator=g).to(BF).cuda()
    seq = torch.tensor([0, 3, -1, 1, 2, 0, 2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([1, 0, 0, 64, 3, 2 ** 31 - 1, 20], dtype=torch.int32, device="cuda")
    t[2, 0] = c.desc.n_pages
    t[2, 1] = -3
    K0, V0 = c.K.clone(), c.V.clone()
    out = torch.full((T, 4, 64), 3.0, dtype=BF, device="cuda")
    c.append(k, v, pos, t, seq=seq, q=qt, q_out=out, freqs=hhr.rope_freqs(64)[0])
    assert c.status() == hhr.HHR_ERR_BAD_INDEX
    pos2 = torch.where(torch.arange(T, device="cuda") == 0, pos, -1)
    check_append(c, K0, V0, k, v, pos2, t, seq, qt, out, hhr.rope_freqs(64)[0])
    assert bool((out[1:] == 3.0).all())
    assert c.status() == hhr.HHR_OK


@pytest.mark.gpu
def test_append_checks():
    c, q, t = make(2, 8, 2, 64, 16, 6)
    k = torch.zeros(2, 2, 64, dtype=BF, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    f = hhr.rope_freqs(64)[0]
    for bad in (dict(k=k[:, :1]), dict(v=k[:1]), dict(k=k.half()), dict(positions=pos.long()), dict(positions=pos[:1]),
                dict(seq=pos[:1]), dict(rope_positions=pos.float()), dict(q=q[:1]), dict(q=q[:, :4]), dict(q_out=q),
                dict(freqs=f.float()), dict(q=q, q_out=q[:1]), dict(freqs=f.cpu())):
        a = dict(k=k, v=k, positions=pos)
        a.update(bad)
        with pytest.raises(ValueError):
            c.append(a.pop("k"), a.pop("v"), a.pop("positions"), t, **a)
    with pytest.raises(hhr.HhrError):
        c.append(k, k, pos, t, freqs=torch.zeros(33, dtype=torch.float64, device="cuda"))
    with pytest.raises(hhr.HhrError):       # three tokens of two sequences need seq
        c.append(k[:1].expand(3, 2, 64), k[:1].expand(3, 2, 64), pos[:1].repeat(3), t)


# ---------------------------------------------------------------- the calls together

@pytest.mark.gpu
@pytest.mark.parametrize("kv,layout,page", [(BF, "head", 16), (BF, "token", 5), (E4, "head", 32)])
def test_decode_steps(kv, layout, page):
    """A prompt, then steps of rotate, store and attend, against the definition over the tokens as they went in."""
    scales = (2.0 ** -4, 2.0 ** -4) if kv == E4 else (1.0, 1.0)
    B, Hq, Hkv, d = 3, 8, 2, 64
    c, _, t = make(B, Hq, Hkv, d, page, 200 // page + 1, kv=kv, layout=layout, scales=scales)
    g = torch.Generator().manual_seed(11)
    f = hhr.rope_freqs(d, base=1e4)[0]
    counts = [150, 0, 33]
    seq = torch.cat([torch.full((n,), i) for i, n in enumerate(counts)]).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(n) for n in counts]).to(torch.int32).cuda()
    k, v = (torch.randn(sum(counts), Hkv, d, generator=g).to(BF).cuda() for _ in range(2))
    c.append(k, v, pos, t, seq=seq, freqs=f)
    lens = torch.tensor(counts, dtype=torch.int32, device="cuda")
    for step in range(4):
        rows = torch.randn(B, Hq + 2 * Hkv, d, generator=g).to(BF).cuda()
        q, kn, vn = rows.split([Hq, Hkv, Hkv], dim=1)
        K0, V0 = c.K.clone(), c.V.clone()
        qr = c.append(kn, vn, lens, t, q=q, freqs=f)
        check_append(c, K0, V0, kn, vn, lens, t, None, q, qr, f, scales=scales)
        lens = lens + 1
        run(c, qr, t, lens.tolist(), scales=scales, name=f"step {step}")


@pytest.mark.gpu
def test_captured_decode_step_follows_lengths_and_tables():
    B, Hq, Hkv, d = 3, 8, 2, 128
    c, _, t = make(B, Hq, Hkv, d, 16, 20)
    f = hhr.rope_freqs(d)[0]
    rows = torch.zeros(B, Hq + 2 * Hkv, d, dtype=BF, device="cuda")
    lens = torch.tensor([5, 0, 100], dtype=torch.int32, device="cuda")
    after = torch.empty_like(lens)
    out = torch.empty(B, Hq, d, device="cuda")

    def step():
        q, k, v = rows.split([Hq, Hkv, Hkv], dim=1)
        qr = c.append(k, v, lens, t, q=q, freqs=f)
        torch.add(lens, 1, out=after)
        c.attend(qr, t, after, out=out)
        return qr

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr = step()
    g = torch.Generator().manual_seed(12)
    for new in ([5, 0, 100], [6, 1, 101], [318, 200, 0], [17, 15, 16]):
        rows.copy_(torch.randn(rows.shape, generator=g).to(BF))
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        t.copy_(t[:, torch.randperm(20, generator=g)])
        K0, V0 = c.K.clone(), c.V.clone()
        graph.replay()
        torch.cuda.synchronize()
        q, k, v = rows.split([Hq, Hkv, Hkv], dim=1)
        check_append(c, K0, V0, k, v, lens, t, None, q, qr, f)
        compare(out, None, attend64(c, qr, t, after))
    assert c.status() == hhr.HHR_OK


@pytest.mark.gpu
def test_two_streams_with_their_own_workspaces():
    c, q, t = make(2, 8, 2, 128, 16, 700)
    lens = torch.tensor([11200, 8000], dtype=torch.int32, device="cuda")
    want = c.attend(q, t, lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [c.new_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for s, w in zip(streams, spaces):
            with torch.cuda.stream(s):
                outs.append(c.attend(q, t, lens, workspace=w))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert [c.status(workspace=w) for w in spaces] == [hhr.HHR_OK] * 2


@pytest.mark.gpu
def test_two_threads_with_tables_of_their_own():
    """Two Python threads on one cache, with tables of different widths: each call has its own description."""
    import threading
    c, q, t = make(2, 8, 2, 64, 16, 60)
    tables, lens = (t[:, :20].contiguous(), t), ([320, 37], [960, 500])
    want, got, bad = [], [[], []], []
    for tab, n in zip(tables, lens):
        want.append(c.attend(q, tab, torch.tensor(n, dtype=torch.int32, device="cuda")).clone())
    spaces = [c.new_workspace() for _ in range(2)]
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()) as _:
                n = torch.tensor(lens[i], dtype=torch.int32, device="cuda")
                for _ in range(200):
                    got[i].append(c.attend(q, tables[i], n, workspace=spaces[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 - reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [x.start() for x in threads]
    [x.join() for x in threads]
    assert not bad, bad
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


@pytest.mark.gpu
def test_hhr_cache_append_and_dense_attention():
    """The retrieval cache takes unrotated tokens: rotated and stored, encoded as hhr_encode_keys does, and its keys and
    values serve attention with a length for each sequence."""
    B, Hq, Hkv, d, cap = 2, 8, 2, 128, 512
    c = hhr.HHRCache(batch=B, q_heads=Hq, kv_heads=Hkv, capacity=cap, P=8, k=64)
    g = torch.Generator().manual_seed(13)
    c.R.copy_(torch.linalg.qr(torch.randn(Hkv, d, d, generator=g))[0])
    c.W.copy_(torch.randn(c.W.shape, generator=g))
    f = hhr.rope_freqs(d, base=1e6)[0]
    paged, table = c.paged()
    paged.head_major = True
    at = 0
    for n in (300, 1, 1):
        rows = torch.randn(B, n, Hq + 2 * Hkv, d, generator=g).to(BF).cuda()
        q, k, v = rows.split([Hq, Hkv, Hkv], dim=2)
        K0, V0 = c.K.clone(), c.V.clone()
        qr = c.append(k, v, at, q=q, freqs=f)
        pos = torch.arange(at, at + n, dtype=torch.int32, device="cuda").repeat(B)
        seq = torch.arange(B, device="cuda").repeat_interleave(n)
        check_append(paged, K0, V0, k.flatten(0, 1), v.flatten(0, 1), pos, table, seq, q.flatten(0, 1), qr.flatten(0, 1), f)
        at += n
    assert qr.shape == (B, 1, Hq, d)
    codes, meta = c.codes.clone(), c.meta.clone()
    c.codes.zero_(), c.meta.zero_()
    c.encode(0, at)
    assert torch.equal(codes, c.codes) and torch.equal(meta, c.meta)
    out = c.decode_step(qr[:, 0].contiguous(), at)
    assert bool(torch.isfinite(out).all()) and c.status() == hhr.HHR_OK
    run(paged, qr[:, 0], table, [at, 17], out_dtype=F32)
    dense = c.dense_attend(qr[:, 0].contiguous(), at)
    mine = paged.attend(qr[:, 0], table, torch.full((B,), at, dtype=torch.int32, device="cuda"), out=torch.empty_like(dense))
    tol = attend64(paged, qr[:, 0], table, torch.full((B,), at))[2]      # each is within it
    assert bool(((mine - dense).abs().cpu() <= 2 * tol + 2.0 ** -23).all())
    for bad in (dict(k=k[:1], v=v[:1]), dict(n_begin=cap), dict(n_begin=-1), dict(k=k[0])):
        a = dict(k=k, v=v, n_begin=0)
        a.update(bad)
        with pytest.raises(ValueError):
            c.append(a["k"], a["v"], a["n_begin"])
