"""GPU parity of attention over a cache of 8 bits with the fp64 oracle of the values it
holds: head sizes, groups, types, pages and blocks, lengths, windows, caps, sinks,
layouts, long histories, slots and scales that no sequence holds, NaN, scores that
outgrow their references; and the whole run: append, chunks, decode, read back."""

import math

import numpy as np
import pytest
import torch

import attention_util as au
from oracle import attention as oatt
from oracle import quantised
from test_gpu_attention_shares import dense_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn


def lib():
    import paged_recurrent_state_amd as m
    m.load()
    return m


def scale_of(top):
    m, e = torch.frexp(top)
    return torch.ldexp(torch.ones_like(top), e - 9 + (m > 0.875))


class Batch:
    """Codes and scales of normal values, and the values they stand for; slots that no sequence holds and scales of
    blocks that none reaches are NaN."""

    def __init__(self, lens, page, block, H, D, seed, heads_first=False, gain=1.0):
        c = au.batch(lens, page, H, D, torch.float32, seed, gain=gain)
        self.lens, self.block = lens, block
        self.args, self.values = {}, {}
        for n in ("k", "v"):
            x = c[n + "_cache"].reshape(-1, page // block, block, H, D)
            top = x.abs().nan_to_num(0.0).amax(dim=(2, 4))
            # (a scale need not be the least that does)
            s = scale_of(top) * 2.0 ** torch.randint(0, 3, top.shape, generator=torch.Generator().manual_seed(seed))
            codes = (x / s[:, :, None, :, None]).to(E4M3)
            self.values[n] = (codes.double() * s.double()[:, :, None, :, None]).reshape(-1, page, H, D)
            s = torch.where(top > 0, s, math.nan)
            codes = codes.view(torch.uint8).reshape(-1, page, H, D)
            if heads_first:
                codes, s = (y.transpose(1, 2).contiguous().transpose(1, 2) for y in (codes, s))
            self.args[n + "_cache"], self.args[n + "_scale"] = codes.to(DEV).view(E4M3), s.to(DEV)
        self.where = {n: c[n].to(DEV) if torch.is_tensor(c[n]) else c[n]
                      for n in ("page_indices", "page_indptr", "page_size", "last_page_len")}

    def oracle(self, q, cu, **kw):
        w = self.where
        return oatt.attention_paged(au.f64(q), cu, self.values["k"].numpy(), self.values["v"].numpy(), w["page_indices"].tolist(),
                                    w["page_indptr"].tolist(), w["page_size"], w["last_page_len"].tolist(), **kw)

    def plain(self, dtype):
        """The same cache in 16 bits."""
        return dict(self.where, **{n + "_cache": self.values[n].to(dtype).to(DEV) for n in "kv"})


def check_chunk(new, past, page, block, H, G, D, dtype, seed, heads_first=False, gain=1.0, same=True, **kw):
    b = Batch([x + y for x, y in zip(new, past)], page, block, H, D, seed, heads_first)
    q = au.queries(sum(new), H * G, D, dtype, seed + 1, DEV, gain)
    cu = [0] + np.cumsum(new).tolist()
    o, lse = lib().attention_prefill_paged(q, au.i32(cu, DEV), **b.args, **b.where, return_lse=True, **kw)
    torch.cuda.synchronize()
    au.check_attention(o, lse, b.oracle(q, cu, **kw), D, dtype, kw.get("softcap", 0.0))
    # the products, their order and the parts are those of a cache in 16 bits
    o2, lse2 = lib().attention_prefill_paged(q, au.i32(cu, DEV), **b.plain(dtype), return_lse=True, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def check_decode(lens, page, block, H, G, D, dtype, seed, heads_first=False, **kw):
    b = Batch(lens, page, block, H, D, seed, heads_first)
    q = au.queries(len(lens), H * G, D, dtype, seed + 1, DEV)
    o, lse = lib().attention_decode_paged(q, **b.args, **b.where, return_lse=True, **kw)
    torch.cuda.synchronize()
    au.check_attention(o, lse, b.oracle(q, None, **kw), D, dtype, kw.get("softcap", 0.0))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_chunk_heads_and_types(D, dtype, G):
    check_chunk([70, 1, 0, 33], [5, 130, 64, 0], 16, 16, 2, G, D, dtype, 100 + D + G)


@pytest.mark.parametrize("page,block", [(16, 16), (48, 16), (48, 48), (96, 32), (128, 128), (896, 64), (896, 896)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages_and_blocks(page, block, D):
    check_chunk([100, 40], [300, 1000], page, block, 2, 2, D, BF, 200 + page + block)
    check_decode([400, 1040, 1, 17], page, block, 2, 3, D, HF, 210 + page + block)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_chunk_lengths(n):
    check_chunk([n], [0], 64, 32, 1, 2, 128, BF, 300 + n)
    check_chunk([n], [n], 48, 16, 1, 1, 256, BF, 310 + n)
    check_chunk([3], [n], 48, 16, 1, 1, 64, HF, 320 + n)


@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 0), (64, 3), (65, 70), (200, 1), (100000, 5), (3, 1000)])
@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (256, BF)])
def test_windows_and_sinks(window, sinks, D, dtype):
    check_chunk([130, 40], [300, 5], 48, 16, 2, 2, D, dtype, 400 + window, window=window, sinks=sinks)
    check_decode([430, 45, 1, 0, 100], 48, 16, 2, 2, D, dtype, 410 + window, window=window, sinks=sinks)


@pytest.mark.parametrize("cap", [0.5, 30.0, 100.0])
@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (256, BF)])
def test_caps(cap, D, dtype):
    check_chunk([100], [200], 32, 32, 2, 2, D, dtype, 500, gain=4.0, softcap=cap)
    check_decode([300, 20], 32, 32, 2, 2, D, dtype, 501, softcap=cap)


@pytest.mark.parametrize("heads_first", [False, True])
def test_layouts(heads_first):
    check_chunk([100, 7], [200, 0], 64, 16, 3, 2, 128, BF, 600, heads_first=heads_first)
    check_decode([300, 7, 0, 64], 64, 16, 3, 2, 128, BF, 601, heads_first=heads_first)
    check_chunk([60], [100], 64, 16, 3, 2, 128, HF, 602, heads_first=heads_first, causal=False)


@pytest.mark.parametrize("G", [1, 5, 16, 17, 40])
def test_decode_groups(G):
    check_decode([70, 1, 0, 33, 500], 64, 64, 2, G, 128, BF, 700 + G)


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, HF), (256, BF)])
def test_decode_long_and_many(D, dtype):
    check_decode([9000], 128, 64, 1, 2, D, dtype, 800)
    check_decode([(i * 37) % 150 for i in range(200)], 16, 16, 2, 2, D, dtype, 801)


def test_many_short_sequences():
    new = [(i * 5) % 7 for i in range(400)]
    check_chunk(new, [(i * 3) % 50 for i in range(400)], 16, 16, 1, 2, 64, BF, 900)


@pytest.mark.parametrize("D,dtype,page,H,cap", [(128, BF, 896, 2, 0.0), (256, HF, 16, 2, 0.0), (64, HF, 48, 2, 20.0)])
def test_long_shares(D, dtype, page, H, cap):
    """More keys a share than places are staged at a time (1,024 of 16 or 8 rows)."""
    new, past, G, block = 800, 56001 if D < 256 else 16001, 12, 16
    L = new + past
    pages = -(-L // page)
    gen = torch.Generator(device=DEV).manual_seed(page + D)
    ids = torch.randperm(pages, generator=gen, device=DEV)
    args, dense = {}, []
    for n in "kv":
        x = torch.randn(pages, page // block, block, H, D, generator=gen, device=DEV)
        s = scale_of(x.abs().amax(dim=(2, 4)))
        codes = (x / s[:, :, None, :, None]).to(E4M3)
        dense.append((codes.float() * s[:, :, None, :, None]).view(pages * page, H, D)[:L].to(dtype))
        codes = codes.view(torch.uint8).view(pages * page, H, D)
        codes[L:] = 0x7f
        paged, scales = torch.empty_like(codes).view(pages, page, H, D), torch.empty_like(s)
        paged[ids], scales[ids] = codes.view(pages, page, H, D), s
        args[n + "_cache"], args[n + "_scale"] = paged.view(E4M3), scales
    q = torch.randn(new, H * G, D, generator=gen, device=DEV).to(dtype)
    o, lse = lib().attention_prefill_paged(q, au.i32([0, new], DEV), **args, page_indices=ids.to(torch.int32),
                                           page_indptr=au.i32([0, pages], DEV), page_size=page,
                                           last_page_len=au.i32([L - (pages - 1) * page], DEV), return_lse=True, softcap=cap)
    torch.cuda.synchronize()
    au.check_attention(o, lse, dense_of(q, *dense, past, cap), D, dtype, cap)


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (256, BF)])
def test_scores_that_outgrow_their_references(D, dtype):
    """Keys that grow with their place: the share is computed again, and gives what a 16-bit cache gives."""
    b = Batch([400], 64, 16, 1, D, 1000)
    grow = torch.arange(400).view(25, 16) // 16
    codes = torch.ones(b.values["k"].shape, dtype=torch.float32)
    ids, page = b.where["page_indices"].tolist(), 64
    scale = torch.ones(len(codes), 4, 1)
    for j in range(25):
        scale[ids[j // 4], j % 4] = 2.0 ** (j // 4 - 3)
    b.args["k_cache"] = codes.to(E4M3).to(DEV)
    b.args["k_scale"] = scale.to(DEV)
    b.values["k"] = codes.double() * scale.double().repeat_interleave(16, dim=1)[..., None]
    assert grow.max() == 24
    q = torch.full((80, 2, D), 8.0 * (128 / D) ** 0.5, dtype=dtype, device=DEV) * (1 + torch.rand(80, 2, 1, device=DEV)).to(dtype)
    o, lse = lib().attention_prefill_paged(q, au.i32([0, 80], DEV), **b.args, **b.where, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, b.oracle(q, [0, 80]), D, dtype)
    q1 = q[-1:].contiguous()
    o, lse = lib().attention_decode_paged(q1, **b.args, **b.where, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, b.oracle(q1, None), D, dtype)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (256, BF)])
def test_nan_reaches_the_rows_that_see_it(which, D, dtype):
    lens, new = [200, 90], [100, 30]
    b = Batch(lens, 48, 16, 2, D, 1100)
    page, off = int(b.where["page_indices"][3]), 150 - 144  # token 150 of the first sequence
    b.args[which + "_cache"].view(torch.uint8)[page, off, 1, 5] = 0x7f
    q = au.queries(130, 4, D, dtype, 1101, DEV)
    cu = [0, 100, 130]
    for window in (0, 20):
        o, lse = lib().attention_prefill_paged(q, au.i32(cu, DEV), **b.args, **b.where, return_lse=True, window=window)
        torch.cuda.synchronize()
        pos = torch.arange(100, 200)
        sees = (pos >= 150) & ((pos < 150 + window) | (window == 0))
        bad = torch.isnan(o.cpu())
        assert not bad[100:].any() and not bad[:, :2].any() and not bad[:100][~sees].any()
        if which == "v":
            assert bad[:100, 2:][sees][..., 5].all() and bad[:100, 2:][sees].sum() == 2 * sees.sum() and torch.isfinite(lse).all()
        else:
            assert bad[:100, 2:][sees].all()
    o, lse = lib().attention_decode_paged(q[:2].contiguous(), **b.args, **b.where, return_lse=True)
    torch.cuda.synchronize()
    bad = torch.isnan(o.cpu())
    assert not bad[1].any() and not bad[0, :2].any()
    assert bad[0, 2:, 5].all() if which == "v" else bad[0, 2:].all()
    assert which == "k" or bad.sum() == 2


def test_codes_past_32_bits():
    """A history on pages that lie over 2^31 codes apart."""
    H, D, page = 8, 128, 64
    b = Batch([200, 70], page, 16, H, D, 1200)
    pages = 40000
    far = torch.tensor([39999, 3, 39000, 20000, 35000, 1], dtype=torch.int64)
    ids = b.where["page_indices"].long().cpu()
    big = {}
    for n in "kv":
        c = torch.zeros(pages, page, H, D, dtype=torch.uint8, device=DEV)
        s = torch.full((pages, 4, H), math.nan, device=DEV)
        c[far.to(DEV)] = b.args[n + "_cache"].view(torch.uint8)[ids.to(DEV)]
        s[far.to(DEV)] = b.args[n + "_scale"][ids.to(DEV)]
        big[n + "_cache"], big[n + "_scale"] = c.view(E4M3), s
    q = au.queries(90, 16, D, BF, 1201, DEV)
    cu = [0, 60, 90]
    where = dict(b.where, page_indices=far.to(torch.int32).to(DEV))
    o, lse = lib().attention_prefill_paged(q, au.i32(cu, DEV), **big, **where, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, b.oracle(q, cu), D, BF)
    q = q[:2].contiguous()
    o, lse = lib().attention_decode_paged(q, **big, **where, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, b.oracle(q, None), D, BF)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    r = np.random.default_rng(seed)
    D, dtype = int(r.choice([64, 128, 256])), [BF, HF][int(r.integers(2))]
    page = int(r.choice([16, 32, 48, 64, 96, 896]))
    block = int(r.choice([n for n in (16, 32, 48, 64, 896) if page % n == 0]))
    B = int(r.integers(1, 6))
    kw = dict(window=int(r.choice([0, 0, 5, 100])), softcap=float(r.choice([0.0, 20.0])), sinks=int(r.choice([0, 2, 40])))
    new, past = [int(x) for x in r.integers(0, 120, B)], [int(x) for x in r.integers(0, 400, B)]
    H, G = int(r.integers(1, 4)), int(r.integers(1, 6))
    check_chunk(new, past, page, block, H, G, D, dtype, 2000 + seed, bool(r.integers(2)), causal=bool(r.integers(4)), **kw)
    check_decode(past, page, block, H, G, D, dtype, 2100 + seed, bool(r.integers(2)), **kw)


def test_streams_workspaces_and_graphs():
    m = lib()
    b = Batch([500, 300, 40], 64, 32, 2, 128, 3000)
    q, cu = au.queries(60, 8, 128, BF, 3001, DEV), au.i32([0, 30, 40, 60], DEV)
    q1 = au.queries(3, 8, 128, BF, 3002, DEV)
    size = m.attention_workspace_size(60, 3, 8, 2, 128)
    ws = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    kw = dict(window=100, sinks=4, return_lse=True)

    def both(i):
        return (*m.attention_prefill_paged(q, cu, **b.args, **b.where, workspace=ws[i], **kw),
                *m.attention_decode_paged(q1, **b.args, **b.where, workspace=ws[i], **kw))

    want = both(0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(both(i))
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(a, c) for a, c in zip(x, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both(0)
    for i in range(3):
        q.copy_(au.queries(60, 8, 128, BF, 3010 + i, DEV))
        q1.copy_(au.queries(3, 8, 128, BF, 3020 + i, DEV))
        b.where["last_page_len"].copy_(au.i32([60 - i, 10 + i, 40 - i], DEV))
        g.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in out]
        # (the first sequence's last tokens lie in slots that hold NaN, which is not equal to itself)
        for a, c in zip(kept, both(1)):
            assert torch.equal(torch.isnan(a), torch.isnan(c)) and torch.equal(a.nan_to_num(7.0), c.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_chunks_decode_and_read(dtype):
    """A run as a program makes it: prompts normed, turned, quantised and attended in chunks, tokens decoded; the
    cache read back is what attention saw."""
    m = lib()
    H, G, D, page, block = 2, 3, 128, 64, 16
    steps = [[70, 33], [64, 0], [1, 1], [1, 1], [13, 50]]
    total = [sum(s[b] for s in steps) for b in range(2)]
    pages = [-(-n // page) for n in total]
    ids = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(1)).tolist()
    lists = [ids[:pages[0]], ids[pages[0]:]]
    cache = [torch.full((sum(pages), page, H, D), 0x7f, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    scale = [torch.full((sum(pages), page // block, H), math.nan, device=DEV) for _ in range(2)]
    tab = m.rope_table(200, 64)
    wq, wk = torch.rand(D, device=DEV) + 0.5, torch.rand(D, device=DEV) + 0.5
    held = [0, 0]
    more = dict(k_scale=scale[0], v_scale=scale[1])
    for i, new in enumerate(steps):
        held = [h + n for h, n in zip(held, new)]
        use = [x[:-(-h // page)] for x, h in zip(lists, held)]
        where = (au.i32(sum(use, []), DEV), au.i32([0, len(use[0]), len(use[0]) + len(use[1])], DEV), page,
                 au.i32([(h - 1) % page + 1 for h in held], DEV))
        T = sum(new)
        q, k, v = au.queries(T, H * (G + 2), D, dtype, 10 + i, DEV).split([H * G, H, H], dim=1)
        cu = None if new == [1, 1] else au.i32([0, new[0], T], DEV)
        q = m.kv_append_paged(k, v, cu, *cache, *where, table=tab, q=q, q_norm=wq, k_norm=wk, **more)
        kw = dict(window=50, sinks=3, return_lse=True, **more)
        o, lse = m.attention_decode_paged(q, *cache, *where, **kw) if cu is None else m.attention_prefill_paged(q, cu, *cache, *where, **kw)
        kb, vb = m.kv_read_paged(au.i32([0, held[0], sum(held)], DEV), sum(held), *cache, *where, **more, dtype=torch.float32)
        torch.cuda.synchronize()
        t = 0
        for b in range(2):
            n, lo = new[b], 0 if b == 0 else held[0]
            for h in range(H):
                kk, vv = au.f64(kb[lo:lo + held[b], h]), au.f64(vb[lo:lo + held[b], h])
                for g in range(G):
                    x = au.f64(q[t:t + n, h * G + g])
                    ref = oatt.softmax_rows(x, kk, vv, range(held[b] - n, held[b]), window=50, sinks=3)
                    au.check_attention(o[t:t + n, h * G + g], lse[t:t + n, h * G + g], ref, D, dtype)
            t += n
    assert quantised.scale_of(1.0) == 2.0 ** -8
