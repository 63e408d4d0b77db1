"""Cases of the attention layers' operators on a paged key/value cache: rotary
positions, the append that rotates on the way, attention of a chunk of new
tokens, and attention of one token per sequence.

A hybrid model runs these beside the recurrent layers, on the same kind of page
table (CSR: ``page_indptr``, ``page_indices``, ``last_page_len``), so the pages
(16 to 1024 tokens, 896 as in the hybrid step among them), batches and lengths
follow those of the recurrent layers' workloads.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the package's entry points on the same inputs.  ``exact``
computes it from the definition in 64 bits, one sequence and head at a time.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}

# A case's fields.  op: "rope" (rotary positions), "rope_grad" (their
# gradient), "append", "chunk", "decode".  seqs sequences with up to `new` new
# and `past` earlier tokens each (lens 0: exactly that many; otherwise the seed
# of ragged lengths).  kv_heads heads in the cache, `group` query heads on each,
# of `dim` values; `page` tokens a page; heads_first: the cache's pages are
# [heads, tokens, dim] instead of [tokens, heads, dim].  rot: rotated values of
# a head; pairs: "half" (i, i + rot/2) or "neighbours" (2i, 2i + 1).  window:
# how many last tokens a token sees (0: all).  softcap: the bound of the tanh on
# the scores (0: none).
BASE = dict(op="chunk", dtype="bf16", seqs=1, new=1, past=0, lens=0, kv_heads=8, group=4, dim=128,
            page=64, heads_first=False, rot=0, pairs="half", window=0, softcap=0.0)


def _case(name, **fields):
    return dict(BASE, name=name, **fields)


def listed():
    return [
        # the rotation of one decoded token in a small model: launch latency
        _case("rope one token", op="rope", kv_heads=2, group=8, dim=256, rot=64, past=2047),
        # the backward pass of the rotation over a training batch of 8 x 4096 tokens
        _case("rope gradient", op="rope_grad", seqs=8, new=4096, rot=128, pairs="neighbours"),
        # the hybrid step's 512 decoded tokens, rotated and written to 896-token pages
        _case("append step", op="append", seqs=512, past=8192, lens=11, page=896, rot=64),
        # prompts of a prefill batch written to small pages, heads first, interleaved pairs
        _case("append prompts", op="append", dtype="fp16", seqs=32, new=4096, past=2048, lens=12, page=16,
              heads_first=True, rot=128, pairs="neighbours"),
        # a few drafted tokens of one request over a short history: latency
        _case("chunk short", new=17, past=1000, page=16),
        # a ragged batch with a window and capped scores, odd pages, heads first
        _case("chunk ragged", dtype="fp16", seqs=8, new=700, past=5000, lens=13, kv_heads=4, group=3, dim=64,
              page=48, heads_first=True, window=1024, softcap=30.0),
        # one step of a long prompt fed in chunks: 2,048 tokens over 32,768
        _case("chunk long", new=2048, past=32768, page=896),
        # a whole prompt at once, 16,384 tokens: the compute-bound case
        _case("chunk whole", new=16384, kv_heads=4),
        # wide heads: four ragged prompts, 16 query heads on 2
        _case("chunk wide", seqs=4, new=3000, past=3000, lens=14, kv_heads=2, group=8, dim=256, page=896),
        # one request, a short history: latency
        _case("decode one", op="decode", past=776, kv_heads=2, group=8, dim=256, page=16),
        # four requests of 131,072 tokens: too few rows to fill the chip without splitting the history
        _case("decode long", op="decode", seqs=4, past=131071),
        # the hybrid step's 512 sequences with mixed histories
        _case("decode step", op="decode", seqs=512, past=4095, lens=15, page=896),
    ]


# What the largest listed case may cost, and what the plain form may hold.
MOST_WORK = 2.2e10           # max(bytes, flops / 50)
MOST_SCORES = 5 * 10 ** 9    # scores of all heads
MOST_GATHERED = 3 * 10 ** 9  # values of the gathered keys


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "append", "append", "chunk", "chunk", "chunk", "decode", "decode", "decode"])
    while True:
        c = dict(BASE, op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]))
        c["kv_heads"] = rng.choice([1, 2, 3, 4, 5, 8, 16])
        c["group"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        c["lens"] = rng.randrange(1, 1 << 20)
        c["page"] = rng.choice([1, 5, 16, 32, 48, 64, 100, 128, 256, 896, 1024])
        c["heads_first"] = rng.random() < 0.4
        c["pairs"] = rng.choice(["half", "neighbours"])
        if op in ("rope", "rope_grad", "append"):
            c["dtype"] = rng.choice(["bf16", "fp16", "fp32"]) if op != "append" else c["dtype"]
            c["dim"] = rng.choice([64, 128, 256] if op == "append" else [64, 80, 96, 128, 256])
            c["rot"] = rng.choice([c["dim"], c["dim"] // 2, c["dim"] // 4])
            c["seqs"] = _log(rng, 1, 512)
            c["new"] = _log(rng, 1, 4096)
            c["past"] = rng.choice([0, _log(rng, 1, 8192)])
        else:
            c["dim"] = rng.choice([64, 128, 256])
            c["softcap"] = rng.choice([0.0, 0.0, 0.0, 30.0, 50.0])
            c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
            c["seqs"] = _log(rng, 1, 512 if op == "decode" else 16)
            c["new"] = _log(rng, 1, 8192) if op == "chunk" else 1
            c["past"] = _log(rng, 1, 65536 if op == "decode" else 32768)
        if 3072 in (c["kv_heads"] * c["dim"], c["kv_heads"] * c["group"] * c["dim"], c["new"], c["past"], c["new"] + c["past"],
                    c["window"]):
            continue
        new, past = _lengths(c)
        heads = c["kv_heads"] * c["group"]
        scores = len(new) * heads * max(new) * max(a + b for a, b in zip(new, past)) if op in ("chunk", "decode") else 0
        pool = sum(a + b for a, b in zip(new, past)) * c["kv_heads"] * c["dim"] if "rope" not in op else 0
        padded = len(new) * max(a + b for a, b in zip(new, past)) * c["kv_heads"] * c["dim"] if op in ("chunk", "decode") else 0
        w = work(c)
        if (max(w["bytes"], w["flops"] / 50) <= MOST_WORK and scores <= MOST_SCORES and max(pool, padded) <= MOST_GATHERED
                and sum(new) * (heads + 2 * c["kv_heads"]) * c["dim"] <= 1.3e9):
            return c


# ------------------------------------------------------------------ lengths

def _lengths(c):
    """New and earlier tokens of each sequence, by the case alone.  Decode adds one
    token to each; "append" with new = 1 is a decode step too."""
    B = c["seqs"]
    if not c["lens"]:
        return [c["new"]] * B, [c["past"]] * B
    rng = random.Random(c["lens"])
    new, past = [], []
    for b in range(B):
        n = c["new"] if c["new"] == 1 else _log(rng, 1, c["new"])
        if c["new"] > 1 and B > 2 and b % 7 == 3:
            n = 0  # a padded sequence
        new.append(n)
        past.append(_log(rng, 1, c["past"] + 1) - 1 if rng.random() < 0.5 else rng.randint(0, c["past"]))
    b = rng.randrange(B)
    if c["new"] > 1:
        new[b] = c["new"]
    past[b] = c["past"]
    return new, past


def _seen(c, n, p):
    """(keys read, (query, key) pairs) of one head of a sequence of n new tokens after p."""
    if not n:
        return 0, 0
    w = c["window"] or (n + p)
    first = max(0, p + 1 - w)
    short = min(max(w - p, 0), n)  # tokens that still see everything before them
    pairs = short * p + short * (short + 1) // 2 + (n - short) * w
    return n + p - first, pairs


def work(c):
    size, D, Hk = BYTES[c["dtype"]], c["dim"], c["kv_heads"]
    Hq = Hk * c["group"]
    new, past = _lengths(c)
    T = sum(new)
    if c["op"] in ("rope", "rope_grad"):
        return {"bytes": 2 * T * (Hq + Hk) * D * size + T * (4 * c["rot"] + 8), "flops": 3 * T * (Hq + Hk) * c["rot"]}
    if c["op"] == "append":
        return {"bytes": 2 * T * (Hq + 2 * Hk) * D * size + T * 4 * c["rot"], "flops": 3 * T * (Hq + Hk) * c["rot"]}
    seen = [_seen(c, n, p) for n, p in zip(new, past)]
    return {"bytes": 2 * sum(k for k, _ in seen) * Hk * D * size + 2 * T * Hq * D * size + 4 * T * Hq,
            "flops": 4 * D * Hq * sum(k for _, k in seen)}


# ------------------------------------------------------------------- inputs

def _randn(gen, *shape, dtype=torch.float32, gain=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32 if dtype == torch.float32 else dtype) * gain)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _table(positions, rot):
    """cos and sin of every position's angles, [positions, rot]: cos, then sin; 64 bits, rounded once."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, D, Hk, ps = DTYPES[c["dtype"]], c["dim"], c["kv_heads"], c["page"]
    Hq = Hk * c["group"]
    new, past = _lengths(c)
    T, B = sum(new), len(new)
    s = {"case": c, "new": new, "past": past, "most_new": max(new), "most_len": max(a + b for a, b in zip(new, past))}
    lengths = [a + b for a, b in zip(new, past)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu_seqlens"] = _i32(cu)
    if c["rot"]:
        s["table"] = _table(s["most_len"], c["rot"])
    if c["op"] in ("rope", "rope_grad"):
        # q and k as they come out of one projection: views of its output
        qkv = _randn(gen, T, Hq + 2 * Hk, D, dtype=dt)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        s["positions"] = torch.cat([torch.arange(p, p + n, device=DEV) for n, p in zip(new, past)])
        return s

    pages = [-(-n // ps) for n in lengths]
    total = sum(pages)
    indptr = [0]
    for n in pages:
        indptr.append(indptr[-1] + n)
    spare = 3
    s["page_indptr"] = _i32(indptr)
    s["page_indices"] = torch.randperm(total + spare, generator=gen, device=DEV)[:total].to(torch.int32)
    s["last_page_len"] = _i32([n - (k - 1) * ps if k else 0 for n, k in zip(lengths, pages)])
    shape = (2, total + spare, Hk, ps, D) if c["heads_first"] else (2, total + spare, ps, Hk, D)
    kv = _randn(gen, *shape, dtype=dt)
    s["k_cache"], s["v_cache"] = (x.transpose(1, 2) if c["heads_first"] else x for x in kv)
    if c["op"] == "append":
        qkv = _randn(gen, T, Hq + 2 * Hk, D, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    else:
        # scores with a spread of 2: some keys stand out, as in a trained model
        s["q"] = _randn(gen, T, Hq, D, dtype=dt, gain=2.0)
    return s


# --------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, pairs, rot):
    """x [T, H, D] in 32 bits; cos, sin [T, rot/2]."""
    cos, sin = cos[:, None], sin[:, None]
    if pairs == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        parts = [a * cos - b * sin, b * cos + a * sin]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        parts = [torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)]
    return torch.cat(parts + [x[..., rot:]], dim=-1)


def _plain_rope(s):
    c = s["case"]
    rows = s["table"][s["positions"]]
    cos, sin = rows[:, :c["rot"] // 2], rows[:, c["rot"] // 2:]
    if c["op"] == "rope_grad":
        sin = -sin
    return [_rotate(s[n].float(), cos, sin, c["pairs"], c["rot"]).to(s[n].dtype) for n in ("q", "k")]


def _token_places(s):
    """Sequence and position of every new token."""
    cu, ptr, lpl = (s[n].long() for n in ("cu_seqlens", "page_indptr", "last_page_len"))
    ps = s["case"]["page"]
    T = s["q"].shape[0]
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True)
    length = (ptr[1:] - ptr[:-1] - 1) * ps + lpl
    return b, t - cu[1:][b] + length[b]


def _plain_append(s):
    c = s["case"]
    ps = c["page"]
    b, pos = _token_places(s)
    rows = s["table"][pos]
    cos, sin = rows[:, :c["rot"] // 2], rows[:, c["rot"] // 2:]
    q, k = (_rotate(s[n].float(), cos, sin, c["pairs"], c["rot"]).to(s[n].dtype) for n in ("q", "k"))
    page = s["page_indices"].long()[s["page_indptr"].long()[b] + pos // ps]
    s["k_cache"][page, pos % ps] = k
    s["v_cache"][page, pos % ps] = s["v"]
    return [q, s["k_cache"], s["v_cache"]]


def _plain_attention(s):
    c = s["case"]
    ps, Hk, G, D, dt = c["page"], c["kv_heads"], c["group"], c["dim"], s["q"].dtype
    B, N, L = c["seqs"], s["most_new"], s["most_len"]
    cu, ptr, lpl = (s[n].long() for n in ("cu_seqlens", "page_indptr", "last_page_len"))
    length = ((ptr[1:] - ptr[:-1] - 1) * ps + lpl)[:, None]
    j = torch.arange(L, device=DEV)
    here = j < length
    page = s["page_indices"].long()[torch.where(here, ptr[:-1, None] + j // ps, 0)]
    off = torch.where(here, j % ps, 0)
    # queries padded to [B, kv heads, tokens x group, D]
    n = (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(N, device=DEV)
    real = i < n
    q = s["q"][torch.where(real, cu[:-1, None] + i, 0)].float()
    q = q.view(B, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B * Hk, N * G, D)
    pos = length - n + i
    seen = (j <= pos[..., None]) & here[:, None]
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    kt = s["k_cache"][page, off].float().permute(0, 2, 3, 1).reshape(B * Hk, D, L)
    x = torch.bmm(q, kt).mul_(1.0 / math.sqrt(D))
    del kt
    if c["softcap"]:
        x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    x = x.view(B, Hk, N, G, L).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True).clamp_(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(dim=-1, keepdim=True)
    v = s["v_cache"][page, off].float().permute(0, 2, 1, 3).reshape(B * Hk, L, D)
    o = torch.bmm(x.view(B * Hk, N * G, L), v).view(B, Hk, N, G, D) / total
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(B, N, Hk * G, D), lse.permute(0, 2, 1, 3).reshape(B, N, Hk * G)
    b, at = torch.nonzero(real, as_tuple=True) if c["op"] == "chunk" else (slice(None), 0)
    return [o[b, at].to(dt), lse[b, at]]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return _plain_rope(s) if "rope" in op else _plain_append(s) if op == "append" else _plain_attention(s)
    import paged_recurrent_state_amd as gdn

    near = c["pairs"] == "neighbours"
    if op == "rope":
        return list(gdn.rope(s["q"], s["k"], s["table"], s["positions"], interleaved=near))
    if op == "rope_grad":
        return list(gdn.rope_backward(s["q"], s["k"], s["table"], s["positions"], interleaved=near))
    pages = (s["page_indices"], s["page_indptr"], c["page"], s["last_page_len"])
    if op == "append":
        cu = None if c["new"] == 1 else s["cu_seqlens"]
        q = gdn.kv_append_paged(s["k"], s["v"], cu, s["k_cache"], s["v_cache"], *pages, table=s["table"], interleaved=near, q=s["q"])
        return [q, s["k_cache"], s["v_cache"]]
    more = dict(window=c["window"], softcap=c["softcap"], return_lse=True)
    if op == "decode":
        return list(gdn.attention_decode_paged(s["q"], s["k_cache"], s["v_cache"], *pages, **more))
    return list(gdn.attention_prefill_paged(s["q"], s["cu_seqlens"], s["k_cache"], s["v_cache"], *pages, **more))


# -------------------------------------------------------------- 64-bit values

def _turned(x, positions, c, sign):
    """Rows of x turned pair by pair, from the angles of the table's definition: the table holds
    their cos and sin rounded to 32 bits, which is what the operators are given."""
    r = c["rot"]
    f = 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
    ang = positions.double()[:, None, None] * f
    turn = torch.complex(ang.cos().float().double(), sign * ang.sin().float().double())
    y = x.double()
    first, second = (slice(0, r // 2), slice(r // 2, r)) if c["pairs"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    new, past, ps = s["new"], s["past"], c["page"]
    Hk, G, D = c["kv_heads"], c["group"], c["dim"]
    if "rope" in c["op"]:
        sign = -1.0 if c["op"] == "rope_grad" else 1.0
        return [_turned(s[n], s["positions"], c, sign) for n in ("q", "k")]
    ptr, idx = s["page_indptr"].tolist(), s["page_indices"].long()
    where = []
    for b in range(len(new)):
        j = torch.arange(past[b] + new[b], device=DEV)
        where.append((idx[ptr[b]:ptr[b + 1]][j // ps], j % ps))
    if c["op"] == "append":
        pos = torch.cat([torch.arange(p, p + n, device=DEV) for n, p in zip(new, past)])
        q, k = (_turned(s[n], pos, c, 1.0) for n in ("q", "k"))
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        t = 0
        for b, (page, off) in enumerate(where):
            n, p = new[b], past[b]
            kc[page[p:], off[p:]] = k[t:t + n]
            vc[page[p:], off[p:]] = s["v"][t:t + n].double()
            t += n
        return [q, kc, vc]
    o = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    lse = torch.zeros(s["q"].shape[:2], device=DEV, dtype=torch.float64)
    t = 0
    for b, (page, off) in enumerate(where):
        n, p = new[b], past[b]
        if not n:
            continue
        for h in range(Hk):
            k, v = s["k_cache"][page, off, h].double(), s["v_cache"][page, off, h].double()
            for lo in range(0, n, 4096):
                hi = min(n, lo + 4096)
                q = s["q"][t + lo:t + hi, h * G:(h + 1) * G].double()
                x = (q.reshape(-1, D) @ k.t()).view(hi - lo, G, n + p) / math.sqrt(D)
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                i = torch.arange(lo, hi, device=DEV)[:, None, None] + p
                j = torch.arange(n + p, device=DEV)
                hidden = (j > i) | (j <= i - c["window"]) if c["window"] else j > i
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, dim=-1)
                x = (x - z[..., None]).exp()
                o[t + lo:t + hi, h * G:(h + 1) * G] = (x.view(-1, n + p) @ v).view(hi - lo, G, D)
                lse[t + lo:t + hi, h * G:(h + 1) * G] = z
                del x
        t += n
    return [o, lse]
