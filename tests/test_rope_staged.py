"""The rotation and the append where they have rows for the whole card: a thread takes four heads of a token, and rows come
through shared memory a tile ahead (by plain loads where they have no 16-byte accesses).  Definitions and tolerances as in
test_rope.py and test_paged.py."""
import pytest
import torch

import kv_cache_retrieval_b200 as hhr
from test_paged import BF, E4, F32, FP16, make, near
from test_rope import _freqs, _x, built, check, exact  # noqa: F401 - built is a fixture

pytestmark = pytest.mark.gpu


def tokens_for(heads, d, size, wide=True):
    """Tokens that give every SM four blocks of four heads a thread, and an odd number of them."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    step = 256 // (d // (2 * (16 // size if wide else 1)))
    return (step * 16 * sms + heads - 1) // heads // 2 * 2 + 3


@pytest.mark.parametrize("dtype,H,d,rot", [(BF, 40, 128, 128), (BF, 7, 64, 32), (FP16, 5, 256, 64), (F32, 33, 64, 64),
                                           (F32, 6, 128, 120), (BF, 4, 512, 512), (FP16, 9, 48, 48), (BF, 4, 16, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_of_many_rows(dtype, H, d, rot, interleaved):
    T = tokens_for(H, d, torch.finfo(dtype).bits // 8)
    x, f = _x((T, H + 2, d), dtype)[:, 1:1 + H], _freqs(rot)
    pos = torch.randint(0, 1 << 20, (T,), dtype=torch.int32, device="cuda")
    check(hhr.rope(x, pos, f, interleaved=interleaved, mscale=1.25), x, pos, f, interleaved=interleaved, mscale=1.25)
    leaf = x.detach().requires_grad_()
    hhr.rope(leaf, pos, f, interleaved=interleaved).backward(x)
    check(leaf.grad, x, pos, f, interleaved=interleaved, transpose=True)
    before = x.clone()
    hhr.rope(x, pos, f, interleaved=interleaved, out=x)
    check(x, before, pos, f, interleaved=interleaved)
    assert torch.equal(x[..., rot:], before[..., rot:])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotation_of_many_rows_of_any_alignment(dtype):
    H, d = 5, 34
    T = tokens_for(H, d, 2, wide=False)
    flat = _x((T * H * d + 1,), dtype)
    x, f = flat[1:].view(T, H, d), _freqs(30)
    pos = torch.randint(0, 1 << 20, (T,), dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        check(hhr.rope(x, pos, f, interleaved=interleaved), x, pos, f, interleaved=interleaved)


@pytest.mark.parametrize("dtype,kv", [(BF, BF), (FP16, FP16), (BF, E4), (FP16, E4)])
@pytest.mark.parametrize("Hq,Hkv,d,rot,page,layout,wide", [
    (5, 3, 256, 256, 16, "head", True), (32, 8, 128, 64, 20, "token", True), (6, 1, 128, 128, 64, "head", True),
    (0, 4, 256, 128, 16, "token", True), (5, 3, 256, 90, 7, "head", False)])
def test_append_of_many_tokens(dtype, kv, Hq, Hkv, d, rot, page, layout, wide):
    """Keys, values and queries of several sequences' prompts, padding rows and rows without a page among them; no other
    place changes."""
    heads = Hq + 2 * Hkv
    T = tokens_for(heads, d, 2, wide)
    scales = (2.0 ** -4, 2.0 ** -6) if kv == E4 else (1.0, 1.0)
    B = 3
    cols = T // B // page + 2
    c, _, table = make(B, max(Hq, Hkv) // Hkv * Hkv if Hq % Hkv else max(Hq, Hkv), Hkv, d, page, cols, dtype=dtype, kv=kv,
                       layout=layout, scales=scales)
    Hq = c.desc.Hq if Hq else 0
    g = torch.Generator().manual_seed(1)
    rows = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(dtype).cuda()
    q, k, v = rows.split([Hq, Hkv, Hkv], dim=1)
    at = torch.arange(T)
    seq, pos = (at % B).to(torch.int32), (at // B).to(torch.int32)
    pos[5::97] = -1                        # padding
    seq[11::301] = B                       # no sequence
    pos[13::401] = cols * page             # no place
    table[1, 2] = -1                       # no page
    live = (pos >= 0) & (seq < B) & (pos < cols * page)
    live &= ~((seq == 1) & (pos // page == 2))
    assert 0 < int((~live).sum()) < T // 4
    f = hhr.rope_freqs(rot)[0]
    K0, V0 = c.K.clone(), c.V.clone()
    out = torch.full((T, Hq, d), 3.0, dtype=dtype, device="cuda") if Hq else None
    c.append(k, v, pos.cuda(), table, seq=seq.cuda(), q=q if Hq else None, q_out=out, freqs=f, mscale=1.125)
    assert c.status() == hhr.HHR_ERR_BAD_INDEX
    view = (lambda x: x) if layout == "token" else (lambda x: x.transpose(1, 2))
    bits = (lambda x: x.view(torch.uint8)) if kv == E4 else (lambda x: x.view(torch.int16))
    s, p = seq[live].long(), pos[live].long()
    ids, off = table.cpu()[s, p // page].long().cuda(), (p % page).cuda()
    y, mag = exact(k[live.cuda()], pos[live], f, mscale=1.125)
    assert near(view(c.K)[ids, off], y, mag, kv, scales[0])
    assert near(view(c.V)[ids, off], v[live.cuda()].double().cpu(), 0 * mag, kv, scales[1])
    untouched = torch.ones(c.K.shape[0], page, dtype=torch.bool, device="cuda")
    untouched[ids, off] = False
    for now, was in ((c.K, K0), (c.V, V0)):
        assert bool((bits(view(now)) == bits(view(was)))[untouched].all())
    if Hq:
        y, mag = exact(q[live.cuda()], pos[live], f, mscale=1.125)
        assert near(out[live.cuda()], y, mag, dtype, 1.0)
        assert bool((out[~live.cuda()] == 3.0).all())
