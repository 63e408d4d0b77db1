"""GPU parity of the paged attention calls against the fp64 oracle, value by
value within the arithmetic's own bound: head sizes, groups, types, page sizes,
lengths, windows, caps, masks that leave rows empty, stale and non-finite values
in slots no sequence holds, strides, streams, graphs and long caches."""

import numpy as np
import pytest
import torch

import attention_util as au
from oracle import attention as oatt

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def lib():
    import paged_recurrent_state_amd as m
    m.load()
    return m


def oracle_of(q, cu, c, **kw):
    return oatt.attention_paged(au.f64(q), cu, au.f64(c["k_cache"]), au.f64(c["v_cache"]),
                                c["page_indices"].tolist(), c["page_indptr"].tolist(), c["page_size"],
                                c["last_page_len"].tolist(), **kw)


def case(new, past, page, Hk, G, D, dtype, seed, heads_first=False, gain=1.0):
    lens = [a + b for a, b in zip(new, past)]
    c = au.batch(lens, page, Hk, D, dtype, seed, DEV, heads_first=heads_first)
    q = au.queries(sum(new), Hk * G, D, dtype, seed + 1, DEV, gain)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return q, cu, c


def run_prefill(q, cu, c, **kw):
    o, lse = lib().attention_prefill_paged(q, au.i32(cu, DEV), **c, return_lse=True, **kw)
    torch.cuda.synchronize()
    return o, lse


def check_prefill(new, past, page, Hk, G, D, dtype, seed, heads_first=False, gain=1.0, **kw):
    q, cu, c = case(new, past, page, Hk, G, D, dtype, seed, heads_first, gain)
    o, lse = run_prefill(q, cu, c, **kw)
    ref = oracle_of(q, cu, c, **kw)
    return au.check_attention(o, lse, ref, D, dtype, kw.get("softcap", 0.0))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_prefill_heads_and_types(D, dtype, G):
    check_prefill([70, 1, 0, 33], [5, 130, 64, 0], 16, 2, G, D, dtype, 100 + D + G)


@pytest.mark.parametrize("page", [1, 5, 16, 48, 64, 100, 896])
def test_prefill_page_sizes(page):
    check_prefill([40, 129, 2], [300, 0, 63], page, 2, 2, 128, BF, page)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_prefill_lengths_without_history(n):
    check_prefill([n], [0], 16, 1, 1, 64, BF, n)


@pytest.mark.parametrize("past", [0, 1, 62, 63, 64, 65, 127, 128, 500])
def test_prefill_histories(past):
    check_prefill([3, 20], [past, past + 7], 16, 1, 4, 128, HF, past)


@pytest.mark.parametrize("window", [1, 2, 17, 64, 65, 200, 100000])
@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (256, BF)])
def test_prefill_windows(window, D, dtype):
    check_prefill([90, 1, 5], [200, 150, 0], 24, 2, 2, D, dtype, window, window=window)


@pytest.mark.parametrize("cap", [0.5, 30.0])
@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (256, BF)])
def test_prefill_softcap(cap, D, dtype):
    check_prefill([80, 9], [60, 100], 16, 1, 4, D, dtype, 7, gain=6.0, softcap=cap, window=50)


def test_prefill_not_causal():
    check_prefill([80, 9, 200], [60, 100, 0], 16, 2, 2, 128, BF, 8, causal=False)
    check_prefill([80, 9, 200], [60, 100, 0], 16, 2, 2, 64, HF, 9, causal=False, window=40)


def test_prefill_scale_and_sharp_scores():
    check_prefill([50], [400], 16, 1, 2, 128, BF, 10, gain=20.0)           # weights on one or two keys
    check_prefill([50], [400], 16, 1, 2, 128, HF, 11, gain=20.0)
    check_prefill([50], [400], 16, 1, 2, 128, BF, 12, scale=0.001)         # nearly flat
    check_prefill([50], [400], 16, 1, 2, 128, BF, 13, scale=1.0)


def test_prefill_rising_scores_move_the_reference():
    """Keys whose scores grow along the sequence: the running reference moves in every tile."""
    q, cu, c = case([40], [600], 16, 1, 2, 128, BF, 14)
    where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), 16, 0)
    for j, (p, i) in enumerate(where):
        c["k_cache"][p, i] = (q[0, 0].float() * (j / 40.0)).to(BF)
    q[:] = q[0, 0]
    o, lse = run_prefill(q, cu, c)
    au.check_attention(o, lse, oracle_of(q, cu, c), 128, BF)


@pytest.mark.parametrize("heads_first", [False, True])
def test_decode_mixed_lengths(heads_first):
    lens = [1, 2, 0, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000, 0, 31]
    for D, dtype, Hk, G, page in ((64, HF, 2, 3, 16), (128, BF, 2, 4, 5), (256, BF, 1, 8, 64)):
        c = au.batch(lens, page, Hk, D, dtype, 20 + D, DEV, heads_first=heads_first)
        q = au.queries(len(lens), Hk * G, D, dtype, 21 + D, DEV, 2.0)
        o, lse = lib().attention_decode_paged(q, **c, return_lse=True)
        torch.cuda.synchronize()
        au.check_attention(o, lse, oracle_of(q, None, c), D, dtype, what=f"D {D}")
        assert (o[2] == 0).all() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("G", [1, 2, 5, 16, 17, 32, 40])
def test_decode_groups(G):
    lens = [700, 33]
    c = au.batch(lens, 16, 2, 128, BF, 30, DEV)
    q = au.queries(2, 2 * G, 128, BF, 31, DEV, 2.0)
    o, lse = lib().attention_decode_paged(q, **c, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, oracle_of(q, None, c), 128, BF)


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, HF), (256, BF)])
@pytest.mark.parametrize("window,cap", [(1, 0.0), (40, 0.0), (64, 20.0), (500, 0.0)])
def test_decode_window_and_cap(D, dtype, window, cap):
    lens = [1, 40, 41, 64, 300, 513]
    c = au.batch(lens, 24, 2, D, dtype, 40, DEV)
    q = au.queries(len(lens), 4, D, dtype, 41, DEV, 3.0)
    o, lse = lib().attention_decode_paged(q, **c, window=window, softcap=cap, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, oracle_of(q, None, c, window=window, softcap=cap), D, dtype, cap)


def test_decode_long_history_is_split():
    """Few rows over long histories, whatever the split: a long one, and lengths around multiples."""
    lens = [20011, 4096, 1]
    c = au.batch(lens, 256, 2, 128, BF, 50, DEV)
    q = au.queries(3, 8, 128, BF, 51, DEV, 2.0)
    o, lse = lib().attention_decode_paged(q, **c, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, oracle_of(q, None, c), 128, BF)


def test_prefill_long_history_is_split():
    check_prefill([5, 3], [6000, 2500], 64, 2, 4, 128, BF, 52)
    check_prefill([200], [3000], 896, 1, 2, 256, BF, 53)


def test_many_short_sequences():
    new = [(i * 7) % 5 for i in range(150)]
    past = [(i * 13) % 70 for i in range(150)]
    check_prefill(new, past, 16, 1, 2, 64, BF, 54)
    lens = [1 + (i * 11) % 90 for i in range(300)]
    c = au.batch(lens, 16, 1, 128, BF, 55, DEV)
    q = au.queries(300, 2, 128, BF, 56, DEV)
    o, lse = lib().attention_decode_paged(q, **c, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, oracle_of(q, None, c), 128, BF)


def test_decode_equals_prefill_of_one_token():
    lens = [77, 5, 800]
    c = au.batch(lens, 16, 2, 128, BF, 60, DEV)
    q = au.queries(3, 8, 128, BF, 61, DEV)
    ref = oracle_of(q, None, c)
    a = lib().attention_decode_paged(q, **c, return_lse=True)
    b = lib().attention_prefill_paged(q, au.i32([0, 1, 2, 3], DEV), **c, return_lse=True)
    torch.cuda.synchronize()
    for o, lse in (a, b):
        au.check_attention(o, lse, ref, 128, BF)


def test_empty_calls():
    m = lib()
    c = au.batch([5, 0], 16, 2, 64, BF, 62, DEV)
    o = m.attention_prefill_paged(torch.empty(0, 4, 64, dtype=BF, device=DEV), au.i32([0, 0, 0], DEV), **c)
    assert o.shape == (0, 4, 64)
    c = au.batch([], 16, 2, 64, BF, 63, DEV)
    o, lse = m.attention_decode_paged(torch.empty(0, 4, 64, dtype=BF, device=DEV), **c, return_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_strided_rows_and_out():
    """q as a view of a fused projection, out as a view of a larger buffer whose rest stays."""
    new, past, Hk, G, D = [30, 3], [50, 9], 2, 3, 64
    _, cu, c = case(new, past, 16, Hk, G, D, BF, 70)
    qkv = au.queries(33, Hk * G + 2 * Hk, D, BF, 71, DEV)
    q = qkv[:, :Hk * G]
    big = torch.full((33, 2, Hk * G, D), 7.0, dtype=BF, device=DEV)
    m = lib()
    o, lse = m.attention_prefill_paged(q, au.i32(cu, DEV), **c, out=big[:, 1], return_lse=True)
    torch.cuda.synchronize()
    assert o.data_ptr() == big[:, 1].data_ptr() and (big[:, 0] == 7).all()
    au.check_attention(o, lse, oracle_of(q, cu, c), D, BF)


def test_interleaved_keys_and_values():
    """Keys and values interleaved page by page in one allocation."""
    c = au.batch([90, 13], 16, 2, 128, BF, 72, DEV)
    both = torch.stack([c["k_cache"], c["v_cache"]], dim=1)
    c["k_cache"], c["v_cache"] = both[:, 0], both[:, 1]
    q = au.queries(2, 4, 128, BF, 73, DEV)
    o, lse = lib().attention_decode_paged(q, **c, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, oracle_of(q, None, c), 128, BF)


def test_infinite_values_in_seen_slots_reach_the_rows_that_see_them():
    """A row of v with an infinity: rows that see it get it, earlier rows do not (their sequence
    ends before it, so it lies in another sequence's pages or past their end)."""
    c = au.batch([64, 65], 16, 1, 128, BF, 74, DEV)
    where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), 16, 1)
    c["v_cache"][where[64][0], where[64][1], 0, 5] = float("inf")
    q = au.queries(2, 2, 128, BF, 75, DEV)
    o = lib().attention_decode_paged(q, **c)
    torch.cuda.synchronize()
    assert torch.isfinite(o[0]).all()
    assert torch.isposinf(o[1, :, 5]).all()
    rest = torch.cat([o[1, :, :5], o[1, :, 6:]], dim=-1)
    assert torch.isfinite(rest).all()


@pytest.mark.parametrize("D,dtype,window,cap", [(64, HF, 0, 0.0), (128, BF, 0, 0.0), (128, HF, 70, 0.0), (256, BF, 0, 20.0)])
@pytest.mark.parametrize("past", [0, 700])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(D, dtype, window, cap, past):
    """NaN and infinities among the values of new tokens: earlier rows of the same chunk do not see them,
    later ones get the formula's value in their column (inf, -inf, or NaN where both meet)."""
    n, Hk, G = 150, 2, 2
    q, cu, c = case([n], [past], 16, Hk, G, D, dtype, 90 + D)
    ref = oracle_of(q, cu, c, window=window, softcap=cap)
    where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), 16, 0)
    bad = [(40, 0, 3, float("nan")), (41, 0, 9, float("inf")), (77, 0, 9, float("-inf")), (100, 1, D - 1, float("-inf")),
           (149, 1, 0, float("inf"))]
    for tok, h, d, x in bad:
        c["v_cache"][where[past + tok][0], where[past + tok][1], h, d] = x
    o, lse = run_prefill(q, cu, c, window=window, softcap=cap)
    x = au.f64(o)
    clean = np.ones(x.shape, dtype=bool)
    for tok, h, d, v in bad:
        last = n if not window else min(n, tok + window)
        rows = slice(tok, last)
        heads = slice(h * G, (h + 1) * G)
        clean[rows, heads, d] = False
        both = d == 9 and v == float("-inf")
        got = x[rows, heads, d]
        if np.isnan(v):
            assert np.isnan(got).all()
        elif both:
            # tokens 41 and 77 meet in column 9: NaN where a row sees the two, -inf where only the second
            two = 41 + window - tok if window else n
            assert np.isnan(got[:max(two, 0)]).all() and np.isneginf(got[max(two, 0):]).all()
        elif d == 9:
            assert np.isposinf(got[:77 - tok]).all()
        else:
            assert (got == v).all()
    eo, el = au.attention_bounds(ref, D, dtype, cap)
    assert (np.abs(x - ref[0])[clean] <= eo[clean]).all()
    assert (np.abs(au.f64(lse) - ref[1]) <= el).all()


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (128, HF), (256, BF)])
@pytest.mark.parametrize("window", [0, 300])
def test_scores_that_outgrow_the_first_block(D, dtype, window):
    """One late key whose score lies far above all before it, in a row's own share and in another's."""
    q, cu, c = case([60], [2000], 64, 1, 2, D, dtype, 95)
    where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), 64, 0)
    q[:] = q[0, 0]
    p, i = where[1990]
    # |q|^2 is about D: a score of 16 sqrt(D), 128 to 256, against about 1 for the others
    c["k_cache"][p, i, 0] = (q[0, 0].float() * 16).to(dtype)
    o, lse = run_prefill(q, cu, c, window=window)
    au.check_attention(o, lse, oracle_of(q, cu, c, window=window), D, dtype)


def rows_of(ref, keep):
    return tuple(x[keep] for x in ref)


def test_nan_query_or_key_stays_in_its_rows():
    q, cu, c = case([40, 40], [10, 10], 16, 1, 2, 64, BF, 76)
    ref = oracle_of(q, cu, c)
    q2 = q.clone()
    q2[3, 1] = float("nan")
    o, lse = run_prefill(q2, cu, c)
    assert torch.isnan(o[3, 1]).all() and torch.isnan(lse[3, 1])
    keep = torch.ones(80, 2, dtype=torch.bool)
    keep[3, 1] = False
    au.check_attention(o.cpu()[keep], lse.cpu()[keep], rows_of(ref, keep.numpy()), 64, BF)
    where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), 16, 0)
    c["k_cache"][where[30][0], where[30][1], 0] = float("nan")   # token 30: rows 20 .. 39 see it
    o, lse = run_prefill(q, cu, c)
    assert torch.isnan(o[20:40]).all() and torch.isnan(lse[20:40]).all()
    keep = np.r_[0:20, 40:80]
    au.check_attention(o.cpu()[keep], lse.cpu()[keep], rows_of(ref, keep), 64, BF)


def test_other_stream_and_repeated_calls():
    q, cu, c = case([100, 3], [700, 900], 16, 2, 4, 128, BF, 80)
    first, lse1 = run_prefill(q, cu, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = lib().attention_prefill_paged(q, au.i32(cu, DEV), **c, return_lse=True)
    s.synchronize()
    assert torch.equal(o, first) and torch.equal(lse, lse1)
    for _ in range(3):
        o, lse = run_prefill(q, cu, c)
        assert torch.equal(o, first) and torch.equal(lse, lse1)


def test_graph_replays_follow_their_inputs():
    """A captured append, prefill and decode, replayed with new inputs and other lengths in place."""
    m = lib()
    Hk, G, D, page = 2, 4, 128, 16
    lens = [[500, 37], [420, 100], [33, 512]]
    c = au.batch([512, 512], page, Hk, D, BF, 81, DEV)
    lpl, ptr, cu = c["last_page_len"], c["page_indptr"], au.i32([0, 20, 30], DEV)
    ids = c["page_indices"].clone()
    q, qd = au.queries(30, Hk * G, D, BF, 82, DEV), au.queries(2, Hk * G, D, BF, 83, DEV)
    c["k_cache"].nan_to_num_(0.0)
    c["v_cache"].nan_to_num_(0.0)
    ws = torch.empty(max(m.attention_workspace_size(30, 2, Hk * G, Hk, D), 256), dtype=torch.uint8, device=DEV)
    o, od = torch.empty_like(q), torch.empty_like(qd)

    def step():
        m.attention_prefill_paged(q, cu, **c, out=o, workspace=ws)
        m.attention_decode_paged(qd, **c, out=od, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k, ln in enumerate(lens):
        pages = [-(-n // page) for n in ln]
        ptr.copy_(au.i32([0, pages[0], sum(pages)], DEV))
        lpl.copy_(au.i32([n - (p - 1) * page for n, p in zip(ln, pages)], DEV))
        c["page_indices"].copy_(ids.roll(k))
        q.copy_(au.queries(30, Hk * G, D, BF, 90 + k, DEV))
        g.replay()
        torch.cuda.synchronize()
        got, gotd = o.clone(), od.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, o) and torch.equal(gotd, od)
        au.check_attention(got, None, oracle_of(q, cu.tolist(), c), D, BF, what=f"replay {k}")
        au.check_attention(gotd, None, oracle_of(qd, None, c), D, BF, what=f"replay {k}")


def test_cache_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 (and bytes past 2^32) from the cache's start."""
    pages, page, Hk, D = 36000, 64, 8, 128
    kv = torch.empty(2, pages, page, Hk, D, dtype=BF, device=DEV)
    ids = [35999, 3, 34000, 35000]
    gen = torch.Generator(device=DEV).manual_seed(1)
    for p in ids:
        kv[:, p] = torch.randn(2, page, Hk, D, generator=gen, device=DEV).to(BF)
    lens = [150, 64]
    table = dict(page_indices=au.i32(ids, DEV), page_indptr=au.i32([0, 3, 4], DEV), page_size=page,
                 last_page_len=au.i32([22, 64], DEV))
    small = kv[:, ids].contiguous()
    ref_c = dict(k_cache=small[0], v_cache=small[1], page_indices=au.i32([0, 1, 2, 3]),
                 page_indptr=au.i32([0, 3, 4]), page_size=page, last_page_len=au.i32([22, 64]))
    q = au.queries(2, 16, D, BF, 2, DEV)
    o, lse = lib().attention_decode_paged(q, kv[0], kv[1], **table, return_lse=True)
    cu = [0, 20, 30]
    qp = au.queries(30, 16, D, BF, 3, DEV)
    op, lsep = lib().attention_prefill_paged(qp, au.i32(cu, DEV), kv[0], kv[1], **table, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, oracle_of(q, None, ref_c), D, BF)
    au.check_attention(op, lsep, oracle_of(qp, cu, ref_c), D, BF)
    assert lens == [150, 64]


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    r = np.random.default_rng(1000 + seed)
    D, dtype = int(r.choice([64, 128, 256])), [BF, HF][int(r.integers(2))]
    Hk, G = int(r.integers(1, 4)), int(r.integers(1, 9))
    B = int(r.integers(1, 6))
    new = [int(x) for x in r.integers(0, 150, B)]
    past = [int(x) for x in r.integers(0, 400, B)]
    kw = dict(window=int(r.choice([0, 0, 30, 200])), softcap=float(r.choice([0.0, 0.0, 15.0])))
    page = int(r.choice([1, 3, 16, 33, 64, 128]))
    if sum(new) == 0:
        new[0] = 1
    check_prefill(new, past, page, Hk, G, D, dtype, 2000 + seed, bool(r.integers(2)), 2.0, **kw)
    lens = [a + b for a, b in zip(new, past)]
    c = au.batch(lens, page, Hk, D, dtype, 3000 + seed, DEV)
    q = au.queries(B, Hk * G, D, dtype, 3001 + seed, DEV, 2.0)
    o, lse = lib().attention_decode_paged(q, **c, return_lse=True, **kw)
    torch.cuda.synchronize()
    au.check_attention(o, lse, oracle_of(q, None, c, **kw), D, dtype, kw["softcap"])
