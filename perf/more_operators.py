"""Cases of the attention layers' further operators: the norm of queries and keys
with the rotation in the same pass, and its gradient; the append that quantises a
cache to 8 bits as it writes, and the read back; attention over such a cache; and
attention with a window whose first tokens stay visible.

A cache of 8 bits holds e4m3 codes and one scale for each block of tokens of a page
and head, a power of two: the least with which the block's largest value is at most
448.  ``k_scale`` and ``v_scale`` are [pages, page_size / block, kv heads].

``run`` computes a case with elementary torch operations in 32 bits (the weights'
gradients, sums over a million rows, in 64), or, where ``own`` is true, with the
package's entry points on the same inputs.  ``exact`` computes it from the definition
in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6

# A case's fields.  op: "norm" (norm and rotation), "norm_grad" (their gradient),
# "append8" (to an 8-bit cache), "read8" (back from it), "chunk8" and "decode8"
# (attention over it), "chunk" and "decode" (over a cache of the queries' type).
# seqs sequences with up to `new` new and `past` earlier tokens each (lens 0: exactly
# that many; otherwise the seed of ragged lengths); read8 reads the `new` last tokens.
# kv_heads heads in the cache, `group` query heads on each, of `dim` values; `page`
# tokens a page, `block` tokens a scale; heads_first: pages are [heads, tokens, dim].
# rot: rotated values of a head; pairs: "half" (i, i + rot/2) or "neighbours".  norm:
# whether the append norms the queries and keys; offset: what is added to the norm's
# weights; wide: weights in fp32.  window: how many last tokens a token sees (0: all),
# sinks: how many first ones besides.  softcap: the bound of the tanh on the scores.
BASE = dict(op="chunk8", dtype="bf16", seqs=1, new=1, past=0, lens=0, kv_heads=8, group=4, dim=128,
            page=64, block=16, heads_first=False, rot=0, pairs="half", norm=False, offset=0.0, wide=False,
            window=0, sinks=0, softcap=0.0)


def _case(name, **fields):
    return dict(BASE, name=name, **fields)


def listed():
    return [
        # norm and rotation of one decoded token in a small model: launch latency
        _case("norm one token", op="norm", kv_heads=2, group=8, dim=256, rot=64, past=2047, offset=1.0),
        # the backward pass of a training batch of 8 x 4096 tokens
        _case("norm gradient", op="norm_grad", seqs=8, new=4096, rot=128, wide=True),
        # the hybrid step's 512 decoded tokens, normed, rotated and quantised into 896-token pages
        _case("append8 step", op="append8", seqs=512, past=2048, lens=11, page=896, block=64, rot=64, norm=True,
              offset=1.0),
        # prompts of a prefill batch quantised into small pages, heads first, interleaved pairs
        _case("append8 prompts", op="append8", dtype="fp16", seqs=32, new=4096, past=2048, lens=12, block=32,
              heads_first=True, rot=128, pairs="neighbours"),
        # the end of one history read back: latency
        _case("read8 one", op="read8", new=200, past=800, block=64),
        # the histories of a batch read back whole
        _case("read8 batch", op="read8", seqs=32, new=16384, lens=16, page=896, block=128),
        # one request, a short history: latency
        _case("decode8 one", op="decode8", past=776, kv_heads=2, group=8, dim=256, page=16),
        # the hybrid step's 512 sequences with mixed histories
        _case("decode8 step", op="decode8", seqs=512, past=4095, lens=15, page=896, block=64),
        # one step of a long prompt fed in chunks: 2,048 tokens over 32,768
        _case("chunk8 long", new=2048, past=32768, page=896, block=128),
        # a ragged batch with a window, first tokens and capped scores, heads first, pages of three blocks
        _case("chunk8 ragged", dtype="fp16", seqs=8, new=700, past=5000, lens=13, kv_heads=4, group=3, dim=64,
              page=48, heads_first=True, window=1024, sinks=4, softcap=30.0),
        # 256 streams far beyond their window
        _case("decode sinks", op="decode", seqs=256, past=16383, lens=17, window=2048, sinks=4, page=16),
        # prompts fed under a window, odd pages
        _case("chunk sinks", op="chunk", seqs=2, new=3000, past=9000, lens=18, window=2000, sinks=64, page=100),
    ]


# What the largest listed case may cost, and what the plain form may hold.
MOST_WORK = 2.2e10           # max(bytes, flops / 50)
MOST_SCORES = 2 * 10 ** 9    # scores of all heads
MOST_GATHERED = 2 * 10 ** 9  # values of the gathered keys


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "append8", "append8", "read8", "chunk8", "chunk8", "decode8", "decode8",
                     "chunk", "decode"])
    while True:
        c = dict(BASE, op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]))
        c["kv_heads"] = rng.choice([1, 2, 3, 4, 5, 8, 16])
        c["group"] = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        c["lens"] = rng.randrange(1, 1 << 20)
        c["heads_first"] = rng.random() < 0.4
        c["dim"] = rng.choice([64, 128, 256])
        if op in ("chunk", "decode"):
            c["page"] = rng.choice([1, 5, 16, 48, 64, 100, 128, 896])
        else:
            c["page"] = rng.choice([16, 32, 48, 64, 96, 128, 256, 896, 1024])
            c["block"] = rng.choice([n for n in (16, 32, 48, 64, 128, 896) if c["page"] % n == 0])
        if op in ("norm", "norm_grad", "append8"):
            c["pairs"] = rng.choice(["half", "neighbours"])
            c["offset"] = rng.choice([0.0, 1.0])
            c["wide"] = rng.random() < 0.5
            c["norm"] = rng.random() < 0.5
            if op != "append8":
                c["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
                c["dim"] = rng.choice([64, 80, 96, 128, 256])
            c["rot"] = rng.choice([c["dim"], c["dim"] // 2, c["dim"] // 4])
            c["seqs"] = _log(rng, 1, 512)
            c["new"] = _log(rng, 1, 4096)
            c["past"] = rng.choice([0, _log(rng, 1, 8192)])
        elif op == "read8":
            c["seqs"], c["new"], c["past"] = _log(rng, 1, 256), _log(rng, 1, 16384), rng.choice([0, _log(rng, 1, 4096)])
        else:
            c["softcap"] = rng.choice([0.0, 0.0, 0.0, 30.0, 50.0])
            if "8" not in op or rng.random() < 0.4:
                c["window"], c["sinks"] = _log(rng, 1, 4096), rng.choice([0, 1, 4, 16, 100, 1000])
            c["seqs"] = _log(rng, 1, 512 if "decode" in op else 16)
            c["new"] = 1 if "decode" in op else _log(rng, 1, 8192)
            c["past"] = _log(rng, 1, 65536 if "decode" in op else 32768)
        new, past = _lengths(c)
        heads, most = c["kv_heads"] * c["group"], max(a + b for a, b in zip(new, past))
        if "decode" in op and c["window"]:
            most = min(most, c["window"] + c["sinks"])
        attends = "chunk" in op or "decode" in op
        scores = len(new) * heads * max(new) * most if attends else 0
        pool = sum(a + b for a, b in zip(new, past)) * c["kv_heads"] * c["dim"] if "norm" not in op else 0
        padded = len(new) * most * c["kv_heads"] * c["dim"] if attends else 0
        w = work(c)
        if (max(w["bytes"], w["flops"] / 50) <= MOST_WORK and scores <= MOST_SCORES and max(pool, padded) <= MOST_GATHERED
                and sum(new) * (heads + 2 * c["kv_heads"]) * c["dim"] <= 5e8):
            return c


# ------------------------------------------------------------------ lengths

def _lengths(c):
    """New and earlier tokens of each sequence, by the case alone.  One new token each is a decode step."""
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
    w = c["window"]
    if not w:
        return n + p, n * p + n * (n + 1) // 2
    # token t sees min(t + 1, w) last tokens, and of the others the first ones
    reach = w + c["sinks"]
    short = min(max(reach - p, 0), n)  # tokens that still see everything before them
    pairs = short * p + short * (short + 1) // 2 + (n - short) * reach
    begin = max(0, p + 1 - w)
    return n + p - begin + min(begin, c["sinks"]), pairs


def work(c):
    size, D, Hk = BYTES[c["dtype"]], c["dim"], c["kv_heads"]
    Hq = Hk * c["group"]
    new, past = _lengths(c)
    T = sum(new)
    table = 4 * T * c["rot"]
    if c["op"] == "norm":
        return {"bytes": 2 * T * (Hq + Hk) * D * size + table + 8 * T, "flops": 8 * T * (Hq + Hk) * D}
    if c["op"] == "norm_grad":
        return {"bytes": 3 * T * (Hq + Hk) * D * size + table + 8 * T, "flops": 20 * T * (Hq + Hk) * D}
    if c["op"] == "append8":
        return {"bytes": 2 * T * Hq * D * size + 2 * T * Hk * D * (size + 1) + table, "flops": 8 * T * (Hq + 2 * Hk) * D}
    if c["op"] == "read8":
        return {"bytes": 2 * T * Hk * D * (size + 1) + 8 * T * Hk // c["block"], "flops": 2 * T * Hk * D}
    seen = [_seen(c, n, p) for n, p in zip(new, past)]
    kv = 1 if c["op"].endswith("8") else size
    return {"bytes": 2 * sum(k for k, _ in seen) * Hk * D * kv + 2 * T * Hq * D * size + 4 * T * Hq,
            "flops": 4 * D * Hq * sum(k for _, k in seen)}


# ------------------------------------------------------------------- inputs

def _randn(gen, *shape, dtype=torch.float32, gain=1.0):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype) * gain


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _table(positions, rot):
    """cos and sin of every position's angles, [positions, rot]: cos, then sin; 64 bits, rounded once."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


def _scale_of(top):
    """The scale of a block whose largest magnitude is `top`: 448 is 7/8 of 2^9."""
    m, e = torch.frexp(top)
    return torch.ldexp(torch.ones_like(top), (e - 9 + (m > 0.875)).clamp_(min=-100)).masked_fill_(top == 0, 2.0 ** -100)


def _quantised(gen, pages, ps, Hk, D, block):
    """Codes [pages, ps, Hk, D] and scales [pages, ps / block, Hk] of normal values, heads of different spread."""
    codes = torch.empty(pages, ps, Hk, D, device=DEV, dtype=E4M3)
    scale = torch.empty(pages, ps // block, Hk, device=DEV)
    gain = _randn(gen, Hk).mul_(0.5).exp_()[:, None]
    step = max(1, (1 << 26) // (ps * Hk * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = _randn(gen, n, ps // block, block, Hk, D).mul_(gain)
        s = _scale_of(x.abs().amax(dim=(2, 4)))
        scale[p:p + n] = s
        codes[p:p + n] = x.div_(s[:, :, None, :, None]).view(n, ps, Hk, D).to(E4M3)
    return codes, scale


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, D, Hk, ps, op = DTYPES[c["dtype"]], c["dim"], c["kv_heads"], c["page"], c["op"]
    Hq = Hk * c["group"]
    new, past = _lengths(c)
    T = sum(new)
    lengths = [a + b for a, b in zip(new, past)]
    s = {"case": c, "new": new, "past": past, "most_new": max(new), "most_len": max(lengths), "tokens": T}
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu_seqlens"] = _i32(cu)
    if c["rot"]:
        s["table"] = _table(s["most_len"], c["rot"])
    if op in ("norm", "norm_grad", "append8"):
        # q, k and v as they come out of one projection: views of its output
        qkv = _randn(gen, T, Hq + 2 * Hk, D, dtype=dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        for n in ("q_weight", "k_weight"):
            w = 1.0 - c["offset"] + 0.2 * _randn(gen, D)
            s[n] = w if c["wide"] else w.to(dt)
    if "norm" in op:
        s["positions"] = torch.cat([torch.arange(p, p + n, device=DEV) for n, p in zip(new, past)])
        if op == "norm_grad":
            s["dq"], s["dk"] = _randn(gen, T, Hq, D, dtype=dt), _randn(gen, T, Hk, D, dtype=dt)
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
    first = c["heads_first"]
    for n in ("k", "v"):
        if op.endswith("8"):
            x, scale = _quantised(gen, total + spare, ps, Hk, D, c["block"])
            s[n + "_scale"] = scale.transpose(1, 2).contiguous().transpose(1, 2) if first else scale
        else:
            x = _randn(gen, total + spare, ps, Hk, D, dtype=dt)
        s[n + "_cache"] = x.transpose(1, 2).contiguous().transpose(1, 2) if first else x
    if op not in ("append8", "read8"):
        # scores with a spread of 2: some keys stand out, as in a trained model
        s["q"] = _randn(gen, T, Hq, D, dtype=dt, gain=2.0)
    return s


# --------------------------------------------------------------- plain forms

def _turn(x, cos, sin, pairs, rot):
    """x [T, H, D] in 32 bits; cos, sin [T, rot/2]."""
    cos, sin = cos[:, None], sin[:, None]
    if pairs == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        parts = [a * cos - b * sin, b * cos + a * sin]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        parts = [torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)]
    return torch.cat(parts + [x[..., rot:]], dim=-1)


def _angles(s, positions):
    rows = s["table"][positions]
    return rows[:, :s["case"]["rot"] // 2], rows[:, s["case"]["rot"] // 2:]


def _plain_rows(s, name, positions, norm):
    """q or k, normed or not, rotated, in 32 bits."""
    c = s["case"]
    x = s[name].float()
    if norm:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * (s[name + "_weight"].float() + c["offset"])
    return _turn(x, *_angles(s, positions), c["pairs"], c["rot"])


def _plain_norm(s):
    return [_plain_rows(s, n, s["positions"], True).to(s[n].dtype) for n in ("q", "k")]


def _plain_norm_grad(s):
    c = s["case"]
    cos, sin = _angles(s, s["positions"])
    dx, dw = [], []
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_weight"]
        dy = _turn(s["d" + n].float(), cos, -sin, c["pairs"], c["rot"])
        r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
        x = x * r
        dn = dy * (w.float() + c["offset"])
        dx.append((r * (dn - x * (dn * x).mean(dim=-1, keepdim=True))).to(s[n].dtype))
        dw.append((dy * x).sum(dim=(0, 1), dtype=torch.float64).to(w.dtype))
    return dx + dw


def _places(s):
    """Position, page and offset of every new token."""
    cu, ptr, lpl = (s[n].long() for n in ("cu_seqlens", "page_indptr", "last_page_len"))
    ps = s["case"]["page"]
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True)
    length = (ptr[1:] - ptr[:-1] - 1) * ps + lpl
    pos = t - cu[1:][b] + length[b]
    return pos, s["page_indices"].long()[ptr[b] + pos // ps], pos % ps


def _plain_append(s):
    c = s["case"]
    n, Hk, D = c["block"], c["kv_heads"], c["dim"]
    per = c["page"] // n
    pos, page, off = _places(s)
    block = page * per + off // n
    q = _plain_rows(s, "q", pos, c["norm"]).to(s["q"].dtype)
    touched, which = torch.unique(block, return_inverse=True)
    at, sub = touched // per, touched % per
    # rows of a block that were there before
    before = torch.full_like(touched, n).scatter_reduce_(0, which, off % n, "amin")
    slots = torch.arange(n, device=DEV)
    for name in ("k", "v"):
        x = _plain_rows(s, name, pos, c["norm"]) if name == "k" else s["v"].float()
        cache, scales = s[name + "_cache"], s[name + "_scale"]
        top = torch.zeros(len(touched), Hk, device=DEV).scatter_reduce_(0, which[:, None].expand(-1, Hk),
                                                                        x.abs().amax(dim=-1), "amax")
        old = scales[at, sub]
        scale = torch.where(before[:, None] > 0, torch.maximum(old, _scale_of(top)), _scale_of(top))
        rows = (at[:, None], sub[:, None] * n + slots)
        codes = cache.view(torch.uint8)[rows].view(E4M3)
        again = (codes.float() * (old / scale)[:, None, :, None]).to(E4M3)
        codes = torch.where((slots < before[:, None])[:, :, None, None], again.view(torch.uint8), codes.view(torch.uint8))
        codes[which, off % n] = (x / scale[which][..., None]).to(E4M3).view(torch.uint8)
        cache.view(torch.uint8)[rows] = codes
        scales[at, sub] = scale
    return [q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _gathered(s, name, page, off):
    """Keys or values at places, in 32 bits."""
    cache = s[name + "_cache"]
    if name + "_scale" not in s:
        return cache[page, off].float()
    x = cache.view(torch.uint8)[page, off].view(E4M3).float()
    return x.mul_(s[name + "_scale"][page, off // s["case"]["block"]][..., None])


def _plain_read(s):
    _, page, off = _places(s)
    return [_gathered(s, n, page, off).to(DTYPES[s["case"]["dtype"]]) for n in ("k", "v")]


def _plain_attention(s):
    c = s["case"]
    ps, Hk, G, D, dt = c["page"], c["kv_heads"], c["group"], c["dim"], s["q"].dtype
    B, N, w, decode = c["seqs"], s["most_new"], c["window"], "decode" in c["op"]
    cu, ptr, lpl = (s[n].long() for n in ("cu_seqlens", "page_indptr", "last_page_len"))
    length = ((ptr[1:] - ptr[:-1] - 1) * ps + lpl)[:, None]
    j = torch.arange(s["most_len"], device=DEV)[None]
    if decode and w and w + c["sinks"] < s["most_len"]:
        # the first tokens and the window alone; what lies in both counts as the window's
        begin = (length - w).clamp(min=0)
        firsts = torch.arange(c["sinks"], device=DEV)[None].expand(B, -1)
        j = torch.cat([torch.where(firsts < begin, firsts, 1 << 40), begin + torch.arange(w, device=DEV)], dim=1)
    here = j < length
    page = s["page_indices"].long()[torch.where(here, ptr[:-1, None] + j // ps, 0)]
    off = torch.where(here, j % ps, 0)
    L = here.shape[1]
    # queries padded to [B, kv heads, tokens x group, D]
    n = (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(N, device=DEV)
    real = i < n
    q = s["q"][torch.where(real, cu[:-1, None] + i, 0)].float()
    q = q.view(B, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B * Hk, N * G, D)
    pos = (length - n + i)[..., None]
    key = j[:, None]
    seen = (key <= pos) & here[:, None]
    if w:
        seen &= (key > pos - w) | (key < c["sinks"])
    kt = _gathered(s, "k", page, off).permute(0, 2, 3, 1).reshape(B * Hk, D, L)
    x = torch.bmm(q, kt).mul_(1.0 / math.sqrt(D))
    del kt
    if c["softcap"]:
        x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    x = x.view(B, Hk, N, G, L).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True).clamp_(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(dim=-1, keepdim=True)
    v = _gathered(s, "v", page, off).permute(0, 2, 1, 3).reshape(B * Hk, L, D)
    o = torch.bmm(x.view(B * Hk, N * G, L), v).view(B, Hk, N, G, D) / total
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(B, N, Hk * G, D), lse.permute(0, 2, 1, 3).reshape(B, N, Hk * G)
    b, at = (slice(None), 0) if decode else torch.nonzero(real, as_tuple=True)
    return [o[b, at].to(dt), lse[b, at]]


PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "append8": _plain_append, "read8": _plain_read}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return PLAIN.get(op, _plain_attention)(s)
    import paged_recurrent_state_amd as gdn

    near = c["pairs"] == "neighbours"
    if "norm" in op:
        more = dict(eps=EPS, weight_offset=c["offset"], interleaved=near)
        rows = (s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"])
        if op == "norm":
            return list(gdn.norm_rope(*rows, **more))
        return list(gdn.norm_rope_backward(s["dq"], s["dk"], *rows, **more))
    pages = (s["page_indices"], s["page_indptr"], c["page"], s["last_page_len"])
    more = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if op.endswith("8") else {}
    if op == "append8":
        if c["norm"]:
            more.update(q_norm=s["q_weight"], k_norm=s["k_weight"], eps=EPS, norm_offset=c["offset"])
        cu = None if c["new"] == 1 else s["cu_seqlens"]
        q = gdn.kv_append_paged(s["k"], s["v"], cu, s["k_cache"], s["v_cache"], *pages, table=s["table"], interleaved=near,
                                q=s["q"], **more)
        return [q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]
    if op == "read8":
        return list(gdn.kv_read_paged(s["cu_seqlens"], s["tokens"], s["k_cache"], s["v_cache"], *pages,
                                      dtype=DTYPES[c["dtype"]], **more))
    more.update(window=c["window"], sinks=c["sinks"], softcap=c["softcap"], return_lse=True)
    if "decode" in op:
        return list(gdn.attention_decode_paged(s["q"], s["k_cache"], s["v_cache"], *pages, **more))
    return list(gdn.attention_prefill_paged(s["q"], s["cu_seqlens"], s["k_cache"], s["v_cache"], *pages, **more))


# -------------------------------------------------------------- 64-bit values

def _complex_turn(y, positions, c, sign):
    """Rows turned pair by pair, from the angles of the table's definition: the table holds their cos
    and sin rounded to 32 bits, which is what the operators are given."""
    r = c["rot"]
    f = 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
    ang = positions.double()[:, None, None] * f
    by = torch.complex(ang.cos().float().double(), sign * ang.sin().float().double())
    first, second = (slice(0, r // 2), slice(r // 2, r)) if c["pairs"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * by
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _normed(s, name, c):
    x = s[name].double()
    rms = (x.pow(2).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt()
    return x / rms, rms, s[name + "_weight"].double() + c["offset"]


def _to_e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even: 3 fraction bits down to 2^-6, then steps of 2^-9."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), e - 3)
    return torch.round(x / step) * step


def _exact_append(s, c, where):
    new, past, n = s["new"], s["past"], c["block"]
    pos = torch.cat([torch.arange(p, p + m, device=DEV) for m, p in zip(new, past)])
    rows = {}
    for name in ("q", "k"):
        y = s[name].double()
        if c["norm"]:
            y, _, w = _normed(s, name, c)
            y = y * w
        rows[name] = _complex_turn(y, pos, c, 1.0)
    rows["v"] = s["v"].double()
    out = [rows["q"]]
    caches = {m: s[m + "_cache"].float().double() for m in ("k", "v")}
    scales = {m: s[m + "_scale"].double() for m in ("k", "v")}
    t = 0
    for b, (page, off) in enumerate(where):
        p, m = past[b], new[b]
        for lo in range(p // n * n, p + m, n) if m else ():
            # one block: tokens lo .. hi of the sequence, of which those before p were there
            hi, old = min(lo + n, p + m), max(p - lo, 0)
            g, o, sub = page[lo], off[lo:hi], int(off[lo]) // n
            for name in ("k", "v"):
                x = rows[name][t + lo + old - p:t + hi - p]
                need = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(0, 2)) / 448.0)))
                had = scales[name][g, sub].clone()
                to = torch.maximum(had, need) if old else need
                if old:
                    caches[name][g, o[:old]] = _to_e4m3(caches[name][g, o[:old]] * (had / to)[:, None])
                caches[name][g, o[old:]] = _to_e4m3(x / to[:, None])
                scales[name][g, sub] = to
        t += m
    return out + [caches["k"], caches["v"], scales["k"], scales["v"]]


def exact(case, seed):
    c = dict(case)
    op = c["op"]
    new, past = _lengths(c)
    if op == "append8" and sum(-(-n // c["block"]) + 1 for n in new) > 6000:
        return None  # (a block at a time: too many of them)
    s = prepare(c, seed)
    ps, Hk, G, D = c["page"], c["kv_heads"], c["group"], c["dim"]
    if op == "norm":
        out = []
        for n in ("q", "k"):
            y, _, w = _normed(s, n, c)
            out.append(_complex_turn(y * w, s["positions"], c, 1.0))
        return out
    if op == "norm_grad":
        dx, dw = [], []
        for n in ("q", "k"):
            y, rms, w = _normed(s, n, c)
            dy = _complex_turn(s["d" + n].double(), s["positions"], c, -1.0)
            # d/dx of x / rms: the part of the gradient across x, over rms; the norm's eps keeps a rest of the part along it
            along = (dy * w * y).sum(-1, keepdim=True) / D
            dx.append((dy * w - y * along) / rms)
            dw.append((dy * y).flatten(0, 1).sum(0))
        return dx + dw
    ptr, idx = s["page_indptr"].tolist(), s["page_indices"].long()
    where = []
    for b in range(len(new)):
        j = torch.arange(past[b] + new[b], device=DEV)
        where.append((idx[ptr[b]:ptr[b + 1]][j // ps], j % ps))
    if op == "append8":
        return _exact_append(s, c, where)

    def rows(name, page, off, h=slice(None)):
        if name + "_scale" not in s:
            return s[name + "_cache"][page, off][:, h].double()
        codes = s[name + "_cache"].view(torch.uint8)[page, off][:, h].contiguous().view(E4M3)
        return codes.float().double() * s[name + "_scale"][page, off // c["block"]][:, h].double()[..., None]

    if op == "read8":
        return [torch.cat([rows(n, pg[p:], off[p:]) for (pg, off), p in zip(where, past)]) for n in ("k", "v")]
    o = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    lse = torch.zeros(s["q"].shape[:2], device=DEV, dtype=torch.float64)
    t = 0
    for b, (page, off) in enumerate(where):
        n, p = new[b], past[b]
        if not n:
            continue
        at = torch.arange(n + p, device=DEV)
        if n == 1 and c["window"]:
            at = at[(at < c["sinks"]) | (at > p - c["window"])]
        keys, values = rows("k", page[at], off[at]), rows("v", page[at], off[at])
        for h in range(Hk):
            for lo in range(0, n, 4096):
                hi = min(n, lo + 4096)
                q = s["q"][t + lo:t + hi, h * G:(h + 1) * G].double()
                x = (q.reshape(-1, D) @ keys[:, h].t()).view(hi - lo, G, len(at)) / math.sqrt(D)
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                i = torch.arange(lo, hi, device=DEV)[:, None, None] + p
                hidden = at > i
                if c["window"]:
                    hidden = hidden | ((at <= i - c["window"]) & (at >= c["sinks"]))
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, dim=-1)
                x = (x - z[..., None]).exp()
                o[t + lo:t + hi, h * G:(h + 1) * G] = (x.view(-1, len(at)) @ values[:, h]).view(hi - lo, G, D)
                lse[t + lo:t + hi, h * G:(h + 1) * G] = z
                del x
        t += n
    return [o, lse]
