"""The calls over 8-bit caches in layouts, batches and uses beside the usual ones, bit for bit what the usual ones
give: keys, values and scales in one allocation, padded batches, empty sequences at either end, shared pages, views in
and out, one workspace under two graphs."""

import pytest
import torch

import attention_util as au

pytestmark = pytest.mark.gpu
DEV, BF, E4M3 = "cuda", torch.bfloat16, torch.float8_e4m3fn
H, G, D, PAGE, BLOCK = 2, 3, 128, 48, 16
NEW, PAST = [30, 0, 1, 70, 4], [100, 40, 33, 0, 500]


def lib():
    import paged_recurrent_state_amd as m
    return m


def bits(x):
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


def table(new, past, extra=3):
    c = au.batch([a + b for a, b in zip(new, past)], PAGE, 1, 64, BF, 3, DEV, spare=extra)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return {n: c[n] for n in ("page_indices", "page_indptr", "page_size", "last_page_len")}, au.i32(cu, DEV), c["k_cache"].shape[0]


def fill(pages):
    gen = torch.Generator(device=DEV).manual_seed(5)
    codes = [torch.randint(0, 0x7f, (pages, PAGE, H, D), generator=gen, device=DEV, dtype=torch.uint8) for _ in "kv"]
    scales = [2.0 ** -torch.randint(6, 10, (pages, PAGE // BLOCK, H), generator=gen, device=DEV).float() for _ in "kv"]
    return codes, scales


def usual(codes, scales):
    (k, v), (ks, vs) = ([x.clone() for x in y] for y in (codes, scales))
    return dict(k_cache=k.view(E4M3), v_cache=v.view(E4M3), k_scale=ks, v_scale=vs)


def joint(codes, scales, form):
    """Keys and values side by side in one allocation, and their scales in another."""
    dims = {"tokens": (0, 1, 2, 3), "heads": (0, 2, 1, 3)}[form.split()[0]]  # of a page in memory
    axis = {"by page": 1, "by token": 3}[form.split(" ", 1)[1]]

    def lay(xs, order):
        x = torch.stack([y.permute(order) for y in xs], dim=axis).contiguous()
        back = [0] * len(order)
        for i, o in enumerate(order):
            back[o] = i
        return [y.permute(back) for y in x.unbind(axis)]

    k, v = lay(codes, dims)
    ks, vs = lay(scales, dims[:3])
    assert k.stride() == v.stride() and ks.stride() == vs.stride() and not k.is_contiguous()
    return dict(k_cache=k.view(E4M3), v_cache=v.view(E4M3), k_scale=ks, v_scale=vs)


def near(a, b):
    """Outputs (bf16) or sums of the same rows over runs cut elsewhere.  Each output is off by its rounding and its weights',
    2^-8 of the values' magnitude (7 at most: codes up to 448 under scales up to 2^-6) each, and by twice what a score is, D
    2^-24 of 300 at most (sum |q k| / sqrt(D), values and queries up to 7 and 4.5): under 3 2^-8 7 in all; a sum by a score's."""
    return bool(((a.float() - b.float()).abs() <= 2 * (3 * 2.0 ** -8 * 7 if a.dtype == BF else D * 2.0 ** -24 * 300)).all())


def use(cache, where, cu, T, x, **kw):
    """Append, chunks, decode and read back: everything that comes out, the caches included."""
    m = lib()
    q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
    tab, w = m.rope_table(1024, 64, device=DEV), torch.linspace(0.5, 1.5, D, device=DEV)
    out = [m.kv_append_paged(k, v, cu, **cache, **where, table=tab, q=q, q_norm=w, k_norm=w)]
    for more in ({}, dict(window=60, sinks=20, softcap=20.0)):
        out += m.attention_prefill_paged(out[0], cu, **cache, **where, return_lse=True, **more, **kw)
        out += m.attention_decode_paged(out[0][:len(where["last_page_len"])], **cache, **where, return_lse=True, **more, **kw)
    out += m.kv_read_paged(cu, T, **cache, **where)
    return [t.clone() for t in (*out, *(y.contiguous() for y in cache.values()))]


@pytest.mark.parametrize("form", ["tokens by page", "heads by page", "tokens by token", "heads by token"])
def test_one_allocation(form):
    where, cu, pages = table(NEW, PAST)
    codes, scales = fill(pages)
    x = au.queries(sum(NEW), H * G + 2 * H, D, BF, 6, DEV)
    want = use(usual(codes, scales), where, cu, sum(NEW), x)
    got = use(joint(codes, scales, form), where, cu, sum(NEW), x)
    for i, (a, b) in enumerate(zip(want, got)):
        assert torch.equal(bits(a), bits(b)), i


@pytest.mark.parametrize("front,back", [(1, 0), (0, 1), (3, 70)])
def test_empty_sequences_at_the_ends(front, back):
    """The same sequences with others around them that have no new tokens, some of them no page."""
    where, cu, pages = table(NEW, PAST)
    codes, scales = fill(pages + 80)
    T = sum(NEW)
    x = au.queries(T, H * G + 2 * H, D, BF, 7, DEV)
    want, got = usual(codes, scales), usual(codes, scales)
    m = lib()
    ids, ptr, lpl = (where[n].tolist() for n in ("page_indices", "page_indptr", "last_page_len"))
    rest = list(range(pages, pages + 80))
    ptr2, ids2, lpl2, cu2 = [0], [], [], [0]
    for j in range(front + len(NEW) + back):
        b = j - front
        if 0 <= b < len(NEW):
            ids2 += ids[ptr[b]:ptr[b + 1]]
            lpl2.append(lpl[b])
            cu2.append(cu2[-1] + NEW[b])
        else:
            held = j % 2  # (a page with one token, or none)
            ids2 += [rest.pop()] * held
            lpl2.append(held)
            cu2.append(cu2[-1])
        ptr2.append(len(ids2))
    wide = dict(page_indices=au.i32(ids2, DEV), page_indptr=au.i32(ptr2, DEV), page_size=PAGE, last_page_len=au.i32(lpl2, DEV))
    tab = m.rope_table(1024, 64, device=DEV)
    q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
    outs = []
    for cache, w, c in ((want, where, cu), (got, wide, au.i32(cu2, DEV))):
        qo = m.kv_append_paged(k, v, c, **cache, **w, table=tab, q=q)
        outs.append([qo, *m.attention_prefill_paged(qo, c, **cache, **w, window=60, sinks=20, return_lse=True),
                     *m.kv_read_paged(c, T, **cache, **w), *cache.values()])
    for i, (a, b) in enumerate(zip(*outs)):
        if i in (1, 2):  # (shares of the batch's key tiles: other runs are cut)
            assert near(a, b), i
        else:
            assert torch.equal(bits(a), bits(b)), i


def test_no_new_tokens_at_all():
    m = lib()
    where, _, pages = table(NEW, PAST)
    codes, scales = fill(pages)
    cache, cu = usual(codes, scales), au.i32([0] * (len(NEW) + 1), DEV)
    x = torch.empty(0, H, D, dtype=BF, device=DEV)
    m.kv_append_paged(x, x, cu, **cache, **where)
    assert m.attention_prefill_paged(torch.empty(0, H * G, D, dtype=BF, device=DEV), cu, **cache, **where).shape == (0, H * G, D)
    assert m.kv_read_paged(cu, 0, **cache, **where)[0].shape == (0, H, D)
    # rows that no sequence has
    x, kept = au.queries(9, H, D, BF, 8, DEV), torch.full((9, H * G, D), 5.0, dtype=BF, device=DEV)
    m.kv_append_paged(x, x, cu, **cache, **where)
    m.attention_prefill_paged(au.queries(9, H * G, D, BF, 9, DEV), cu, **cache, **where, out=kept)
    back = [torch.full((9, H, D), 5.0, dtype=BF, device=DEV) for _ in "kv"]
    m.kv_read_paged(cu, 9, **cache, **where, k_out=back[0], v_out=back[1])
    torch.cuda.synchronize()
    assert all((y == 5.0).all() for y in (kept, *back))
    for n, want in (("k_cache", codes[0]), ("v_cache", codes[1]), ("k_scale", scales[0]), ("v_scale", scales[1])):
        assert torch.equal(bits(cache[n]), bits(want))


def test_padded_rows_and_views():
    m = lib()
    where, cu, pages = table(NEW, PAST)
    codes, scales = fill(pages)
    T, B = sum(NEW), len(NEW)
    x = au.queries(T + 11, H * G + 2 * H, D, BF, 10, DEV)
    x[T:] = float("nan")
    q = x[:, :H * G]
    cache = usual(codes, scales)
    for more in ({}, dict(window=60, sinks=20)):
        want = m.attention_prefill_paged(q[:T].contiguous(), cu, **cache, **where, **more)
        wide = torch.full((T + 11, H * G + 1, D + 8), 5.0, dtype=BF, device=DEV)
        got = m.attention_prefill_paged(q, cu, **cache, **where, **more, out=wide[:, 1:, :D])
        assert got.data_ptr() == wide[:, 1:].data_ptr()
        torch.cuda.synchronize()
        assert torch.isfinite(want).all() and near(wide[:T, 1:, :D], want)
        assert (wide[T:] == 5.0).all() and (wide[:, 0] == 5.0).all() and (wide[..., D:] == 5.0).all()
        q1 = q[:B].transpose(0, 1).contiguous().transpose(0, 1)
        want = m.attention_decode_paged(q[:B].contiguous(), **cache, **where, **more)
        assert torch.equal(m.attention_decode_paged(q1, **cache, **where, **more, out=q1), want)


def test_sequences_that_share_pages():
    """The same history under several sequences, and one page several times in a history."""
    m = lib()
    codes, scales = fill(6)
    cache = usual(codes, scales)
    q = au.queries(4, H * G, D, BF, 11, DEV)
    q[1:] = q[:1]
    ids = [4, 2, 2, 5]
    shared = dict(page_indices=au.i32(ids * 4, DEV), page_indptr=au.i32([0, 4, 8, 12, 16], DEV), page_size=PAGE, last_page_len=au.i32([7] * 4, DEV))
    copies = [[y[[0, 1, 2, 3, 4, 5] + [2]] for y in z] for z in (codes, scales)]
    alone = dict(page_indices=au.i32([4, 2, 6, 5], DEV), page_indptr=au.i32([0, 4], DEV), page_size=PAGE, last_page_len=au.i32([7], DEV))
    got = m.attention_decode_paged(q, **cache, **shared, return_lse=True)
    want = m.attention_decode_paged(q[:1], **usual(*copies), **alone, return_lse=True)
    for a, b in zip(got, want):
        assert near(a, b.expand_as(a))
    k, v = m.kv_read_paged(au.i32([0, 151, 302, 453, 604], DEV), 604, **cache, **shared)
    assert torch.equal(k[:151], k[151:302]) and torch.equal(v[:151], v[453:]) and torch.equal(k[48:96], k[96:144])


def test_two_graphs_share_a_workspace():
    m = lib()
    where, cu, pages = table(NEW, PAST)
    cache = usual(*fill(pages))
    T, B = sum(NEW), len(NEW)
    q = au.queries(T, H * G, D, BF, 12, DEV)
    ws = torch.empty(m.attention_workspace_size(T, B, H * G, H, D), dtype=torch.uint8, device=DEV)
    calls = [lambda: m.attention_prefill_paged(q, cu, **cache, **where, workspace=ws, window=60, sinks=20),
             lambda: m.attention_decode_paged(q[:B], **cache, **where, workspace=ws)]
    graphs, outs = [], []
    for call in calls:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for i in range(3):
        q.copy_(au.queries(T, H * G, D, BF, 13 + i, DEV))
        for g in graphs if i % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        kept = [o.clone() for o in outs]
        assert all(torch.equal(a, call()) for a, call in zip(kept, calls))
