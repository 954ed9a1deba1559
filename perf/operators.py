"""The measured cases of the serving operators: rotary positions, the append to a paged key-value
cache, and the attention of one new token over it, each in a plain form and through the package."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------
# cases

def _rope(name, T, H, d, rot, dtype, interleaved, scaling, grad, row_heads, max_pos):
    return {"name": name, "op": "rope", "T": T, "H": H, "d": d, "rot": rot, "dtype": dtype, "interleaved": interleaved,
            "scaling": scaling, "grad": grad, "row_heads": row_heads, "max_pos": max_pos}


def _append(name, T, seqs, Hq, Hkv, d, rot, dtype, cache, interleaved, scaling, page, layout, pages, max_pos):
    return {"name": name, "op": "append", "T": T, "seqs": seqs, "Hq": Hq, "Hkv": Hkv, "d": d, "rot": rot, "dtype": dtype,
            "cache": cache, "interleaved": interleaved, "scaling": scaling, "page": page, "layout": layout, "pages": pages,
            "max_pos": max_pos}


def _attend(name, B, Hq, Hkv, d, dtype, cache, out, page, layout, max_len, lens, window):
    return {"name": name, "op": "attend", "B": B, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype, "cache": cache, "out": out,
            "page": page, "layout": layout, "max_len": max_len, "lens": lens, "window": window}


def listed():
    return [
        # the 32 query and 8 key heads of one decode step of eight sequences, far into their contexts
        _rope("rope_step", 8, 40, 128, 128, "bf16", False, "none", False, 40, 131072),
        # a prompt chunk: query and key heads inside the fused projection's rows (their 8 value heads stay), yarn frequencies
        _rope("rope_prompt_yarn", 8192, 40, 128, 128, "bf16", False, "yarn", False, 48, 131072),
        # training in float32 with half of each head rotated, pairs interleaved: output and gradient, an odd number of tokens
        _rope("rope_grad_partial", 4095, 32, 128, 64, "f32", True, "none", True, 32, 4096),
        # one decode step of eight sequences: rotate the queries, rotate and store the keys, store the values
        _append("append_step", 8, 8, 32, 8, 128, 128, "bf16", "bf16", False, "bands", 16, "head", 512, 131072),
        # a large decode batch over an 8-bit cache with pages of 32 tokens, token-major
        _append("append_batch_e4m3", 256, 256, 32, 8, 128, 128, "bf16", "e4m3", False, "linear", 32, "token", 512, 65536),
        # a prompt chunk of five sequences of different lengths, half of each head rotated, an odd number of tokens
        _append("append_prompt", 8191, 5, 32, 8, 128, 64, "f16", "f16", True, "ntk", 16, "head", 1024, 8192),
        # the shortest everyday call: one sequence of some hundred tokens, its last page partly filled
        _attend("attend_short", 1, 32, 8, 128, "bf16", "bf16", "same", 16, "head", 517, "full", 0),
        # one long sequence: the headline context of the retrieval benchmark, float32 output as its dense attention has
        _attend("attend_128k", 1, 32, 8, 128, "bf16", "bf16", "f32", 16, "head", 131072, "full", 0),
        # the batched long-context workload, token-major pages of 32
        _attend("attend_batch8_64k", 8, 32, 8, 128, "bf16", "bf16", "same", 32, "token", 65536, "full", 0),
        # a serving batch of very different lengths, empty sequences among them, groups of eight heads
        _attend("attend_ragged", 61, 64, 8, 128, "f16", "f16", "same", 16, "token", 8191, "ragged", 0),
        # an 8-bit cache, groups of sixteen heads
        _attend("attend_e4m3", 16, 64, 4, 128, "bf16", "e4m3", "same", 64, "head", 32768, "ragged", 0),
        # a sliding window over heads of 64 elements without groups
        _attend("attend_window_d64", 24, 16, 16, 64, "bf16", "bf16", "same", 16, "head", 16000, "ragged", 4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    d = rng.choice([64, 128, 128, 256])
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    rot = rng.choice([d, d, d // 2, d // 4])
    if op == "rope":
        H = rng.randint(1, 48)
        T = _log(rng, 1, max(1, 8192 * 40 * 128 // (H * d) // 4))
        c = _rope("", T, H, d, rot, rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.5, scaling, rng.random() < 0.3,
                  H + rng.choice([0, 0, 1, 8]), _log(rng, 4096, 1 << 20))
    elif op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        T = _log(rng, 1, 4096)
        page = rng.choice([1, 8, 16, 32, 64, 20])
        dtype = rng.choice(["bf16", "f16"])
        seqs = T if rng.random() < 0.5 else rng.randint(1, min(T, 16))
        pages = -(-T // page) + 2 * seqs + rng.randint(1, 64)
        c = _append("", T, seqs, Hq, Hkv, d, rot, dtype, rng.choice([dtype, "e4m3"]), rng.random() < 0.5, scaling, page,
                    rng.choice(["head", "token"]), pages, _log(rng, 8192, 1 << 18))
    else:
        Hkv = rng.choice([1, 2, 4, 8])
        r = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16, 24])
        B = _log(rng, 1, 64)
        most = max(64, 131072 * 8 * 128 // (B * Hkv * d) // 2)
        dtype = rng.choice(["bf16", "f16"])
        c = _attend("", B, Hkv * r, Hkv, d, dtype, rng.choice([dtype, dtype, "e4m3"]), rng.choice(["same", "f32"]),
                    rng.choice([1, 8, 16, 32, 64, 20]), rng.choice(["head", "token"]), _log(rng, 1, min(131072, most)),
                    rng.choice(["full", "ragged"]), rng.choice([0, 0, 0, 128, 1000]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------
# inputs

def _freqs(rot, base, kind, max_pos):
    """Radians per position of each pair, and the factor on the rotated elements (float64, by the published formulas)."""
    half = rot // 2
    j = torch.arange(half, dtype=torch.float64)
    f = base ** (-2.0 * j / rot)
    orig = 4096.0
    factor = max(1.0, max_pos / orig)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "ntk" and rot > 2:
        return (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * j / rot), 1.0
    if kind == "yarn":
        dim = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), half - 1)
        keep = 1.0 - ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    if kind == "bands":
        turns = orig * f / (2 * math.pi)
        s = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f / factor * (1 - s) + f * s, 1.0
    return f, 1.0


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _scale(case, which):
    # what a calibration keeps for an 8-bit cache; powers of two here
    return {"k": 2.0 ** -4, "v": 2.0 ** -6}[which] if case["cache"] == "e4m3" else 1.0


def _pool(g, case, pages, channel, scale):
    """A cache pool filled with what earlier sequences left: per-channel scales with a few outliers for keys."""
    H, d, page = case["Hkv"], case["d"], case["page"]
    shape = (pages, H, page, d) if case["layout"] == "head" else (pages, page, H, d)
    out = torch.empty(shape, dtype=DTYPES[case["cache"]], device="cuda")
    if channel is not None:
        channel = channel[:, None, :] if case["layout"] == "head" else channel
    step = max(1, (64 << 20) // (H * page * d))
    for at in range(0, pages, step):
        x = torch.randn(out[at:at + step].shape, generator=g, device="cuda")
        x = x if channel is None else x * channel
        x = x / scale
        out[at:at + step] = x.clamp(-E4M3_MAX, E4M3_MAX).to(out.dtype) if case["cache"] == "e4m3" else x.to(out.dtype)
    return out


def _channels(g, H, d):
    s = torch.exp(0.5 * torch.randn((H, d), generator=g, device="cuda"))
    s.scatter_(1, torch.rand((H, d), generator=g, device="cuda").topk(4, dim=1).indices,
               8.0 * s.new_ones((H, 4)))
    return s


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] != "attend":
        f, s["mscale"] = _freqs(case["rot"], 500000.0, case["scaling"], case["max_pos"])
        s["freqs"] = f.cuda()
    if case["op"] == "rope":
        T, H, d, dt = case["T"], case["H"], case["d"], DTYPES[case["dtype"]]
        rows = _normal(g, (T, case["row_heads"], d), dt)
        s["x"] = rows[:, :H]
        # consecutive positions of a chunk, or the unrelated ones of a decode batch
        if T > 64:
            first = int(torch.randint(0, max(1, case["max_pos"] - T), (1,), generator=g, device="cuda"))
            s["pos"] = torch.arange(first, first + T, dtype=torch.int32, device="cuda")
        else:
            s["pos"] = torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["out"] = torch.empty((T, H, d), dtype=dt, device="cuda")
        if case["grad"]:
            s["g"] = _normal(g, (T, H, d), dt)
            s["x"] = s["x"].detach().requires_grad_()
    elif case["op"] == "append":
        T, n, page, dt = case["T"], case["seqs"], case["page"], DTYPES[case["dtype"]]
        rows = _normal(g, (T, case["Hq"] + 2 * case["Hkv"], case["d"]), dt)   # the fused projection's rows
        s["q"], s["k"], s["v"] = rows.split([case["Hq"], case["Hkv"], case["Hkv"]], dim=1)
        s["q_out"] = torch.empty((T, case["Hq"], case["d"]), dtype=dt, device="cuda")
        s["K"] = _pool(g, case, case["pages"], _channels(g, case["Hkv"], case["d"]), _scale(case, "k"))
        s["V"] = _pool(g, case, case["pages"], None, _scale(case, "v"))
        # sequence i appends a run of tokens from its present length on
        cuts = sorted(torch.randperm(T - 1, generator=g, device="cuda")[:n - 1].add(1).tolist()) if n > 1 else []
        cuts = [0] + cuts + [T]
        cols = -(-case["max_pos"] // page)
        table = torch.randint(0, case["pages"], (n, cols), generator=g, device="cuda", dtype=torch.int32)
        counts = torch.tensor([b - a for a, b in zip(cuts, cuts[1:])], device="cuda")
        first = (torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * (case["max_pos"] - counts)).long()
        seq = torch.repeat_interleave(torch.arange(n, device="cuda"), counts)
        pos = first[seq] + torch.arange(T, device="cuda") - torch.tensor(cuts[:-1], device="cuda")[seq]
        used = torch.unique(seq * cols + pos // page)     # the pages that are written: pages of their own
        table.view(-1)[used] = torch.randperm(case["pages"], generator=g, device="cuda")[:used.numel()].to(torch.int32)
        s["table"], s["seq"], s["pos"] = table, seq.to(torch.int32), pos.to(torch.int32)
    else:
        B, page, dt = case["B"], case["page"], DTYPES[case["dtype"]]
        s["q"] = _normal(g, (B, case["Hq"], case["d"]), dt)
        lens = torch.full((B,), case["max_len"], dtype=torch.int32, device="cuda")
        if case["lens"] == "ragged":
            u = torch.rand(B, generator=g, device="cuda")
            lens = (u * u * (case["max_len"] + 1)).to(torch.int32).clamp_(max=case["max_len"])
            lens[0], lens[-1] = 0, case["max_len"]
        cols = -(-case["max_len"] // page)
        need = -(-lens.long() // page)
        pages = int(need.sum()) + 3
        s["table"] = torch.zeros((B, cols), dtype=torch.int32, device="cuda")
        inside = torch.arange(cols, device="cuda")[None] < need[:, None]
        s["table"][inside] = torch.randperm(pages, generator=g, device="cuda")[:int(need.sum())].to(torch.int32)
        s["K"] = _pool(g, case, pages, _channels(g, case["Hkv"], case["d"]), _scale(case, "k"))
        s["V"] = _pool(g, case, pages, None, _scale(case, "v"))
        s["lens"] = lens
        s["out"] = torch.empty((B, case["Hq"], case["d"]), dtype=torch.float32 if case["out"] == "f32" else dt, device="cuda")
        s["lse"] = torch.empty((B, case["Hq"]), dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# plain forms

def _rotate(x, pos, freqs, mscale, interleaved, transpose, wide):
    """x [T, H, d] rotated by pos * freqs, in `wide` arithmetic (angles always in 64 bits)."""
    rot = 2 * freqs.numel()
    a = pos.to(torch.float64)[:, None, None] * freqs
    cos, sin = (mscale * torch.cos(a)).to(wide), (mscale * torch.sin(a)).to(wide)
    sin = -sin if transpose else sin
    x = x.to(wide)
    part, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        x1, x2 = part[..., 0::2], part[..., 1::2]
        y = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), dim=-1).flatten(-2)
    else:
        x1, x2 = part[..., :rot // 2], part[..., rot // 2:]
        y = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), dim=-1)
    return torch.cat((y, rest), dim=-1)


def _plain_rope(s):
    c, x = s["case"], s["x"].detach()
    y = _rotate(x, s["pos"], s["freqs"], s["mscale"], c["interleaved"], False, torch.float32).to(x.dtype)
    if not c["grad"]:
        return y
    return y, _rotate(s["g"], s["pos"], s["freqs"], s["mscale"], c["interleaved"], True, torch.float32).to(x.dtype)


def _store(pool, case, page_ids, offsets, rows, scale):
    rows = rows / scale
    rows = rows.clamp(-E4M3_MAX, E4M3_MAX) if case["cache"] == "e4m3" else rows
    rows = rows.to(pool.dtype)
    if case["cache"] == "e4m3":   # the indexed write goes by the bytes
        pool, rows = pool.view(torch.uint8), rows.view(torch.uint8)
    if case["layout"] == "head":
        pool = pool.transpose(1, 2)
    pool[page_ids, offsets] = rows


def _plain_append(s):
    c = s["case"]
    turn = (s["pos"], s["freqs"], s["mscale"], c["interleaved"], False, torch.float32)
    pos, seq = s["pos"].long(), s["seq"].long()
    ids, off = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    _store(s["K"], c, ids, off, _rotate(s["k"], *turn), _scale(c, "k"))
    _store(s["V"], c, ids, off, s["v"].to(torch.float32), _scale(c, "v"))
    return _rotate(s["q"], *turn).to(s["q"].dtype), s["K"], s["V"]


def _rows(pool, case, table, wide):
    """[B, Hkv, tokens, d] of the sequences' pages, in `wide`."""
    x = pool[table.long()] if pool.dtype != torch.float8_e4m3fn else pool.view(torch.uint8)[table.long()].view(pool.dtype)
    x = x.to(wide)
    if case["layout"] == "head":
        x = x.transpose(2, 3)
    B, P, page, H, d = x.shape
    return x.reshape(B, P * page, H, d).transpose(1, 2)


def _softmax_rows(q, K, V, lens, case, wide):
    """(out, lse) of q [B, Hq, d] over the tokens inside each sequence and its window; zeros and -inf for none."""
    B, Hq, d = q.shape
    Hkv = K.shape[1]
    x = torch.matmul(q.to(wide).view(B, Hkv, Hq // Hkv, d), K.transpose(2, 3)) * (_scale(case, "k") / math.sqrt(d))
    n = torch.arange(K.shape[2], device=q.device)[None]
    inside = n < lens[:, None]
    if case["window"]:
        inside = inside & (n >= lens[:, None] - case["window"])
    x = torch.where(inside[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = w.sum(-1, keepdim=True)
    y = torch.matmul(w, V) / torch.where(total > 0, total, 1.0) * _scale(case, "v")
    return y.view(B, Hq, d), (m + torch.log(total)).view(B, Hq)


def _plain_attend(s):
    c = s["case"]
    y, lse = _softmax_rows(s["q"], _rows(s["K"], c, s["table"], torch.float32), _rows(s["V"], c, s["table"], torch.float32),
                           s["lens"], c, torch.float32)
    return y.to(s["out"].dtype), lse


# ---------------------------------------------------------------------------------------------
# the package's calls

def _cache(s):
    if "cache" not in s:   # the handle that a serving program makes once over its pools
        from kv_cache_retrieval_b200 import HHRPagedCache
        c = s["case"]
        s["cache"] = HHRPagedCache(q_heads=c["Hq"], kv_heads=c["Hkv"], page=c["page"], head_dim=c["d"], dtype=DTYPES[c["dtype"]],
                                   layout=c["layout"], K=s["K"], V=s["V"], k_scale=_scale(c, "k"), v_scale=_scale(c, "v"))
    return s["cache"]


def _own_rope(s):
    from kv_cache_retrieval_b200 import rope
    c = s["case"]
    if not c["grad"]:
        return rope(s["x"], s["pos"], s["freqs"], interleaved=c["interleaved"], mscale=s["mscale"], out=s["out"])
    y = rope(s["x"], s["pos"], s["freqs"], interleaved=c["interleaved"], mscale=s["mscale"])
    return y.detach(), torch.autograd.grad(y, s["x"], s["g"])[0]


def _own_append(s):
    q = _cache(s).append(s["k"], s["v"], s["pos"], s["table"], seq=s["seq"], q=s["q"], q_out=s["q_out"], freqs=s["freqs"],
                         interleaved=s["case"]["interleaved"], mscale=s["mscale"])
    return q, s["K"], s["V"]


def _own_attend(s):
    y = _cache(s).attend(s["q"], s["table"], s["lens"], out=s["out"], lse=s["lse"], window=s["case"]["window"])
    return y, s["lse"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attend": _own_attend}[op](state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[op](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    if case["op"] == "rope":
        n = case["T"] * case["H"] * case["d"] * (2 if case["grad"] else 1)
        return {"bytes": 2 * n * SIZES[case["dtype"]] + 4 * case["T"] + 4 * case["rot"],
                "flops": 3 * n * case["rot"] // case["d"]}
    if case["op"] == "append":
        T, Hq, Hkv, d = case["T"], case["Hq"], case["Hkv"], case["d"]
        i, o = SIZES[case["dtype"]], SIZES[case["cache"]]
        return {"bytes": T * d * ((2 * Hq + 2 * Hkv) * i + 2 * Hkv * o) + 12 * T + 4 * case["rot"],
                "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    B, Hq, Hkv, d, n = case["B"], case["Hq"], case["Hkv"], case["d"], case["max_len"]
    w = case["window"] if case["window"] else n
    if case["lens"] == "full":
        tokens = B * min(n, w)
    else:   # the mean of min(u * u * n, w) over u in [0, 1), and one sequence of length n
        u = min(1.0, math.sqrt(w / n))
        tokens = max(B - 2, 0) * (n * u ** 3 / 3 + min(n, w) * (1 - u)) + min(n, w)
    out = 4 if case["out"] == "f32" else SIZES[case["dtype"]]
    return {"bytes": 2 * tokens * Hkv * d * SIZES[case["cache"]] + B * Hq * (d * (SIZES[case["dtype"]] + out) + 4)
            + 4 * tokens / case["page"] + 4 * B, "flops": 4 * tokens * Hq * d}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain forms: complex turns, logsumexp, one sequence at a time

def _turned(x, s, sign):
    f = s["freqs"]
    n, T = f.numel(), x.shape[0]
    z = torch.polar(torch.full((T, 1, n), float(s["mscale"]), dtype=torch.float64, device="cuda"),
                    sign * torch.outer(s["pos"].double(), f)[:, None])
    y = x.detach().double().clone()
    if s["case"]["interleaved"]:
        y[..., :2 * n] = torch.view_as_real(torch.view_as_complex(y[..., :2 * n].reshape(T, -1, n, 2)) * z).flatten(-2)
    else:
        t = torch.complex(y[..., :n].contiguous(), y[..., n:2 * n].contiguous()) * z
        y[..., :n], y[..., n:2 * n] = t.real, t.imag
    return y


def _exact_append(s):
    c = s["case"]
    pools = []
    slot = s["table"].long().reshape(-1)[s["seq"].long() * s["table"].shape[1] + s["pos"].long().div(c["page"], rounding_mode="floor")]
    slot = slot * c["page"] + s["pos"].long().remainder(c["page"])
    for pool, rows, scale in ((s["K"], _turned(s["k"], s, 1.0), _scale(c, "k")), (s["V"], s["v"].double(), _scale(c, "v"))):
        p = pool.double()
        if c["layout"] == "head":
            p = p.transpose(1, 2).contiguous()
        flat = p.view(-1, c["Hkv"], c["d"])
        flat.index_copy_(0, slot, rows / scale)
        pools.append(p.transpose(1, 2).contiguous() if c["layout"] == "head" else p)
    return _turned(s["q"], s, 1.0), pools[0], pools[1]


def _exact_attend(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    out = torch.zeros((B, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n <= lo:
            continue
        at = torch.arange(lo, n, device="cuda")
        ids, off = s["table"][b].long()[at // c["page"]], at % c["page"]
        for h in range(Hkv):
            k, v = (x[ids, h, off] if c["layout"] == "head" else x[ids, off, h]
                    for x in (s["K"].view(torch.uint8) if c["cache"] == "e4m3" else s["K"],
                              s["V"].view(torch.uint8) if c["cache"] == "e4m3" else s["V"]))
            if c["cache"] == "e4m3":
                k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
            r = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = s["q"][b, r].double() @ (k.double() * _scale(c, "k")).T * d ** -0.5
            lse[b, r] = torch.logsumexp(x, -1)
            out[b, r] = torch.exp(x - lse[b, r, None]) @ (v.double() * _scale(c, "v"))
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attend":
        return _exact_attend(s)
    y = _turned(s["x"], s, 1.0)
    return (y, _turned(s["g"], s, -1.0)) if case["grad"] else y
