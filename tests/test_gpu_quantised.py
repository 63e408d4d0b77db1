"""GPU parity of the append to a cache of 8 bits and of the read back with the oracle:
codes and scales exact where no value is computed, within a code's half step where
keys are normed and turned; blocks, pages, layouts, decoded tokens that join a
block, what is stored of odd values, what may not be written, graphs and streams."""

import numpy as np
import pytest
import torch

import attention_util as au
from oracle import attention as oatt
from oracle import norms, quantised

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
E4M3 = torch.float8_e4m3fn
MOST = {BF: 1.875 * 2.0 ** 127, HF: 61440.0}


def lib():
    import paged_recurrent_state_amd as m
    m.load()
    return m


def table_of(lens, page, seed, spare=2):
    gen = torch.Generator().manual_seed(seed)
    pages = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(pages) + spare, generator=gen)[:sum(pages)].to(torch.int32)
    ptr = np.concatenate([[0], np.cumsum(pages)])
    lpl = [n - (k - 1) * page if k else 0 for n, k in zip(lens, pages)]
    return dict(page_indices=ids.to(DEV), page_indptr=au.i32(ptr.tolist(), DEV), page_size=page, last_page_len=au.i32(lpl, DEV))


def codes_of(x):
    """fp64 values of a tensor of codes."""
    return x.contiguous().view(torch.uint8).cpu().view(E4M3).double().numpy()


def same(got, want, what=""):
    assert np.array_equal(got, want, equal_nan=True), f"{what}: {(~((got == want) | (np.isnan(got) & np.isnan(want)))).sum()} differ"


class Cache:
    """Codes and scales of random bits (NaN among them), and the oracle's copy."""

    def __init__(self, lens, page, block, H, D, seed, heads_first=False):
        self.where = table_of(lens, page, seed)
        pages = len(self.where["page_indices"]) + 2
        gen = torch.Generator().manual_seed(seed + 1)
        self.block = block
        self.c, self.s, self.codes, self.scales = {}, {}, {}, {}
        for n in "kv":
            x = torch.randint(0, 256, (pages, page, H, D), generator=gen, dtype=torch.uint8).view(E4M3)
            s = 2.0 ** torch.randint(-20, 3, (pages, page // block, H), generator=gen).float()
            self.codes[n], self.scales[n] = x.double().numpy().copy(), s.double().numpy().copy()
            x, s = x.to(DEV), s.to(DEV)
            if heads_first:
                x, s = (y.view(torch.uint8) if y.dtype == E4M3 else y for y in (x, s))
                x, s = (y.transpose(1, 2).contiguous().transpose(1, 2) for y in (x, s))
                x = x.view(E4M3)
            self.c[n + "_cache"], self.s[n + "_scale"] = x, s

    def append(self, k, v, cu, **kw):
        return lib().kv_append_paged(k, v, cu, **self.c, **self.where, **self.s, **kw)

    def expect(self, name, rows, new, lens, most):
        quantised.append(self.codes[name], self.scales[name], rows, new, lens, self.where["page_indices"].tolist(),
                         self.where["page_indptr"].tolist(), self.where["page_size"], self.block, most)

    def check(self, name, what=""):
        same(self.s[name + "_scale"].cpu().double().numpy(), self.scales[name], f"{what} scales of {name}")
        same(codes_of(self.c[name + "_cache"]), self.codes[name], f"{what} codes of {name}")


def check_exact(new, past, page, block, H, D, dtype, seed, heads_first=False, decode=False, spread=3.0):
    """Keys that do not turn, and values: codes and scales bit for bit, and everything else left as it was."""
    lens = [a + b for a, b in zip(new, past)]
    a = Cache(lens, page, block, H, D, seed, heads_first)
    T = sum(new)
    gen = torch.Generator().manual_seed(seed + 5)
    kv = (torch.randn(T, 2 * H, D, generator=gen) * torch.exp(spread * torch.randn(T, 2 * H, 1, generator=gen))).to(dtype).to(DEV)
    k, v = kv[:, :H], kv[:, H:]
    cu = None if decode else au.i32([0] + np.cumsum(new).tolist(), DEV)
    assert a.append(k, v, cu) is None
    torch.cuda.synchronize()
    for n, x in (("k", k), ("v", v)):
        a.expect(n, au.f64(x), new, lens, MOST[dtype])
        a.check(n)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_types_heads_and_layouts(dtype, D, heads_first):
    check_exact([20, 0, 1, 7, 70], [3, 5, 31, 0, 50], 32, 16, 2, D, dtype, 20 + D, heads_first)


@pytest.mark.parametrize("page,block", [(16, 16), (48, 16), (48, 48), (64, 32), (96, 48), (128, 128), (896, 64), (896, 896), (1024, 16)])
def test_pages_and_blocks(page, block):
    check_exact([9, 130, 1, 4, 5], [60, 0, 895, 11, 27], page, block, 3, 128, BF, 30 + block)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 15, 16, 17, 31, 32, 33, 64, 100, 1000])
@pytest.mark.parametrize("past", [0, 7, 16])
def test_lengths(n, past):
    check_exact([n], [past], 64, 16, 1, 64, BF, 40 + n)


def test_decoded_tokens_join_blocks():
    """One token of each sequence at a time, over the ends of blocks and pages."""
    past = [0, 1, 15, 16, 30, 47, 48, 90]
    H, D, page, block = 2, 128, 48, 16
    steps = 20
    a = Cache([p + steps for p in past], page, block, H, D, 50)
    full = a.where
    gen = torch.Generator().manual_seed(51)
    for s in range(steps):
        lens = [p + s + 1 for p in past]
        lpl = [(n - 1) % page + 1 for n in lens]
        ptr = np.concatenate([[0], np.cumsum([-(-n // page) for n in lens])])
        first = full["page_indptr"].tolist()
        ids = [full["page_indices"].tolist()[first[b]:first[b] - (-n // page)] for b, n in enumerate(lens)]
        a.where = dict(full, page_indices=au.i32(sum(ids, []), DEV), page_indptr=au.i32(ptr.tolist(), DEV), last_page_len=au.i32(lpl, DEV))
        k, v = ((torch.randn(8, H, D, generator=gen) * 2.0 ** (s % 7)).to(BF).to(DEV) for _ in range(2))
        a.append(k, v, None if s % 2 else au.i32(list(range(9)), DEV))
        torch.cuda.synchronize()
        for n, x in (("k", k), ("v", v)):
            a.expect(n, au.f64(x), [1] * 8, lens, MOST[BF])
            a.check(n, f"step {s}")


def test_a_large_block_takes_tokens_late():
    """Over 800 rows rounded to a new scale, by decoded tokens and by a chunk."""
    check_exact([1, 1, 1], [895, 700, 1], 896, 896, 2, 64, BF, 60, decode=True, spread=6.0)
    check_exact([50, 30], [700, 860], 896, 896, 2, 64, BF, 61, spread=6.0)


def test_many_sequences():
    new = [(i * 5) % 7 for i in range(300)]
    check_exact(new, [(i * 13) % 90 for i in range(300)], 32, 16, 2, 64, BF, 62)
    check_exact([1] * 300, [(i * 13) % 90 for i in range(300)], 32, 32, 1, 128, HF, 63, decode=True)


@pytest.mark.parametrize("D,block", [(64, 896), (256, 896), (64, 128), (256, 64)])
def test_blocks_of_every_length_among_one_workgroups_tokens(D, block):
    """Sixty-four tokens a workgroup, whose blocks one, two or all of its waves take, or read twice."""
    new = [3, 1, 300, 20, 2, 0, 130, 70, 17, 1100, 5, 40, 9, 33, 257, 64, 128, 16, 1, 1] * 2
    check_exact(new, [(i * 37) % 120 for i in range(len(new))], 896, block, 8, D, HF if D == 64 else BF, 68)


def test_odd_values():
    H, D = 1, 64
    for dtype in (BF, HF):
        a = Cache([16, 16, 16, 16, 16], 16, 16, H, D, 64)
        x = au.queries(80, 2, D, dtype, 65, DEV)
        x[0:16] = 0.0
        x[17, 0, 3], x[18, 1, 5], x[19, 0, 9] = float("nan"), float("inf"), -float("inf")
        x[32:48] = float("nan")
        x[50] = torch.finfo(dtype).max  # the code next to it is beyond the type
        x[51] = -torch.finfo(dtype).max
        x[64:80] = torch.finfo(dtype).tiny * 0.25
        k, v = x[:, :1], x[:, 1:]
        a.append(k, v, au.i32([0, 16, 32, 48, 64, 80], DEV))
        torch.cuda.synchronize()
        for n, y in (("k", k), ("v", v)):
            a.expect(n, au.f64(y), [16] * 5, [16] * 5, MOST[dtype])
            a.check(n, str(dtype))
        back = lib().kv_read_paged(au.i32([0, 16, 32, 48, 64, 80], DEV), 80, **a.c, **a.where, **a.s, dtype=dtype)
        assert torch.isfinite(back[0][48:64]).all() and torch.isnan(back[0][17, 0, 3]) and torch.isnan(back[1][18, 0, 5])


def test_more_tokens_than_the_table_holds_writes_none_of_the_excess():
    a = Cache([4], 16, 16, 2, 64, 66)
    kv = au.queries(6, 4, 64, BF, 67, DEV)
    a.append(kv[:, :2], kv[:, 2:], au.i32([0, 6], DEV))
    torch.cuda.synchronize()
    for n, x in (("k", kv[:, :2]), ("v", kv[:, 2:])):
        a.expect(n, au.f64(x)[2:], [4], [4], MOST[BF])
        a.check(n)
    back = lib().kv_read_paged(au.i32([0, 6], DEV), 6, **a.c, **a.where, **a.s)
    assert (back[0][:2] == 0).all() and (back[1][:2] == 0).all()


@pytest.mark.parametrize("new", [[1, 2, 0, 1], [40, 3, 0, 7]])
@pytest.mark.parametrize("normed,coded", [(True, False), (False, True), (True, True)])
def test_rows_behind_the_last_sequence_stay(new, normed, coded):
    m, past, H, D, page, block = lib(), [5, 0, 3, 16], 2, 64, 32, 16
    lens, T = [a + b for a, b in zip(new, past)], sum(new)
    tab = m.rope_table(64, 32, device=DEV)
    cu = au.i32([0] + np.cumsum(new).tolist(), DEV)
    k, v, q = (au.queries(T + 9, h, D, BF, 70 + i, DEV) for i, h in enumerate((H, H, 6)))
    w = torch.ones(D, device=DEV) if normed else None

    def run(rows):
        a = Cache(lens, page, block, H, D, 73)
        kv = a.c if coded else {n: torch.full(c.shape, 7.0, dtype=BF, device=DEV) for n, c in a.c.items()}
        out = torch.full((T + 9, 6, D), 3.0, dtype=BF, device=DEV)
        m.kv_append_paged(k[:rows], v[:rows], cu, **kv, **a.where, **(a.s if coded else {}), table=tab, q=q[:rows], q_out=out[:rows],
                          q_norm=w, k_norm=w)
        torch.cuda.synchronize()
        return [out, *(x.view(torch.uint8) for x in kv.values()), *(a.s.values() if coded else ())]

    exact, padded = run(T), run(T + 9)
    assert (padded[0][T:] == 3.0).all() and torch.isfinite(padded[0]).all()
    for x, y in zip(exact, padded):
        assert torch.equal(x, y)


def half_step(x):
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 4)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("D,rot,normed", [(128, 128, False), (128, 64, True), (64, 32, True), (256, 64, False), (64, 4, True),
                                          (256, 20, True), (128, 0, True)])
def test_turned_and_normed_keys(dtype, near, D, rot, normed):
    m = lib()
    new, past, Hq, Hk, page, block = [30, 1, 0, 5, 64], [3, 40, 2, 0, 60], 5, 2, 64, 32
    lens = [a + b for a, b in zip(new, past)]
    a = Cache(lens, page, block, Hk, D, 70)
    T = sum(new)
    qkv = au.queries(T, Hq + 2 * Hk, D, dtype, 71, DEV)
    q, k, v = qkv.split([Hq, Hk, Hk], dim=1)
    wq, wk = torch.rand(D, device=DEV) + 0.5, torch.rand(D, device=DEV) + 0.5
    tab = m.rope_table(160, rot) if rot else None
    pos = [p + i for n, p in zip(new, past) for i in range(n)]
    kw = dict(q_norm=wq, k_norm=wk, eps=1e-5, norm_offset=0.25) if normed else {}
    tb = au.f64(tab) if rot else np.zeros((160, 0))

    def want(x, w):
        return norms.norm_rope(au.f64(x), au.f64(w), tb, pos, 1e-5, 0.25, near) if normed else oatt.rotate(au.f64(x), tb, pos, near)

    cu = au.i32([0] + np.cumsum(new).tolist(), DEV)
    qo = a.append(k, v, cu, q=q, table=tab, interleaved=near, **kw)
    torch.cuda.synchronize()
    w = want(q, wq)
    top = np.abs(w).max(axis=-1, keepdims=True) * 2
    u = au.UNIT[dtype]
    assert (np.abs(au.f64(qo) - w) <= top * 2.0 ** -19 * (1 + u) + u * np.abs(w) + au.TINY[dtype]).all()
    a.expect("v", au.f64(v), new, lens, MOST[dtype])
    a.check("v")
    before = a.codes["k"].copy()
    w = want(k, wk)
    a.expect("k", w, new, lens, MOST[dtype])
    scale = a.s["k_scale"].cpu().double().numpy()
    same(scale, a.scales["k"], "scales of k")  # (no block's largest value lies within fp32 rounding of a border)
    got, exp = codes_of(a.c["k_cache"]), a.codes["k"]
    untouched = (before == exp) | (np.isnan(before) & np.isnan(exp))
    # a code is off by half a step of the larger of the two, and by what the value in fp32 is
    lim = np.maximum(half_step(got), half_step(exp)) * 2 + 1e-9
    off = np.abs(got - exp)
    assert ((off <= lim) | (np.isnan(got) & np.isnan(exp))).all()
    # next to no code differs at all: the value would have to lie within 2^-18 of its row's largest of a border
    assert (off[~untouched] > 0).mean() < 1e-3


def test_rows_of_four_bytes_and_strides():
    """Rows that start at multiples of 4 bytes alone; keys and values of one buffer; out over q."""
    m = lib()
    H, D, T = 2, 64, 40
    tab = m.rope_table(64, 64)
    x = au.queries(T, 6, D, BF, 72, DEV)
    flat = torch.empty(T * 6 * D + 2, dtype=BF, device=DEV)
    odd = flat[2:].view(T, 6, D)
    odd.copy_(x)
    outs = []
    for src in (x, odd, x.transpose(0, 1).contiguous().transpose(0, 1)):
        a = Cache([25, 30], 32, 32, H, D, 73)
        q, k, v = src.split([2, 2, 2], dim=1)
        q = q.clone() if src is not odd else q
        qo = a.append(k, v, au.i32([0, 20, 40], DEV), q=q, table=tab, q_out=q)
        torch.cuda.synchronize()
        assert qo.data_ptr() == q.data_ptr()
        outs.append((qo.clone(), codes_of(a.c["k_cache"]), codes_of(a.c["v_cache"]), a.s["k_scale"].clone(), a.s["v_scale"].clone()))
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[3], outs[0][3]) and torch.equal(o[4], outs[0][4])
        same(o[1], outs[0][1])
        same(o[2], outs[0][2])


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_read_back(dtype, D, heads_first):
    lens, H = [20, 0, 1, 95, 200], 3
    a = Cache(lens, 48, 16, H, D, 80, heads_first)
    for n in "kv":  # (scales that keep every value inside fp16)
        a.s[n + "_scale"].fill_(0.125)
        a.s[n + "_scale"][1::2] = 2.0
        a.scales[n] = a.s[n + "_scale"].cpu().double().numpy()
    counts = [20, 0, 1, 40, 150]
    cu = [0] + np.cumsum(counts).tolist()
    kept = torch.full((cu[-1] + 2, H, D), 7.0, dtype=dtype, device=DEV)
    k, v = lib().kv_read_paged(au.i32(cu, DEV), cu[-1] + 2, **a.c, **a.where, **a.s, dtype=dtype, k_out=kept)
    torch.cuda.synchronize()
    assert k.data_ptr() == kept.data_ptr() and (kept[-2:] == 7.0).all(), "rows behind the last sequence changed"
    for name, got in (("k", k), ("v", v)):
        want = []
        for b, n in enumerate(counts):
            where = oatt.slots(a.where["page_indices"].tolist(), a.where["page_indptr"].tolist(),
                               a.where["last_page_len"].tolist(), 48, b)
            want += [a.codes[name][p, i] * a.scales[name][p, i // 16][:, None] for p, i in where[lens[b] - n:]]
        same(au.f64(got[:-2]), np.stack(want), name)
    # one token of each sequence
    k1, _ = lib().kv_read_paged(None, 5, **a.c, **a.where, **a.s, dtype=dtype)
    torch.cuda.synchronize()
    ends = [cu[b + 1] - 1 for b in range(5)]
    for b in (0, 2, 3, 4):
        same(au.f64(k1[b]), au.f64(k[ends[b]]))
    assert (k1[1] == 0).all()


def test_append_then_read_is_within_a_half_step():
    m = lib()
    lens, H, D = [300, 17], 4, 128
    a = Cache(lens, 64, 32, H, D, 81)
    kv = au.queries(317, 2 * H, D, BF, 82, DEV)
    cu = au.i32([0, 300, 317], DEV)
    a.append(kv[:, :H], kv[:, H:], cu)
    k, v = m.kv_read_paged(cu, 317, **a.c, **a.where, **a.s)
    torch.cuda.synchronize()
    for got, x in ((k, kv[:, :H]), (v, kv[:, H:])):
        # 2^-4 of the value, or half the least step, 2^-10 of a scale of at most 2^-6 (values under 448 / 64)
        assert ((got.double() - x.double()).abs() <= x.double().abs() * 2.0 ** -4 + 2.0 ** -16).all()


def test_offsets_past_32_bits():
    m = lib()
    pages, page, H, D = 40000, 64, 8, 128  # 2.6e9 codes
    c = [torch.zeros(pages, page, H, D, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2)]
    s = [torch.ones(pages, 1, H, device=DEV) for _ in range(2)]
    where = (au.i32([39999, 39000, 2], DEV), au.i32([0, 1, 3], DEV), page, au.i32([64, 1], DEV))
    k, v = au.queries(2, H, D, BF, 83, DEV), au.queries(2, H, D, BF, 84, DEV)
    m.kv_append_paged(k, v, None, *c, *where, k_scale=s[0], v_scale=s[1])
    kb, vb = m.kv_read_paged(None, 2, *c, *where, k_scale=s[0], v_scale=s[1])
    torch.cuda.synchronize()
    for got, x in ((kb, k), (vb, v)):
        # the first token joins a block of scale 1 and keeps it: half its least step is 2^-9 / 2
        assert ((got.double() - x.double()).abs() <= x.double().abs() * 2.0 ** -4 + 2.0 ** -10).all()
    assert (c[0].view(torch.uint8)[39999, 63] != 0).any() and (c[1].view(torch.uint8)[2, 0] != 0).any()


def test_graph_replays_and_other_streams():
    m = lib()
    a, H, D = Cache([41, 30], 32, 16, 2, 128, 85), 2, 128
    qkv = au.queries(2, 8, D, BF, 86, DEV)
    q, k, v = qkv.split([4, 2, 2], dim=1)
    tab, qo = m.rope_table(64, 128), torch.empty(2, 4, D, dtype=BF, device=DEV)
    w = torch.rand(D, device=DEV)
    cu = au.i32([0, 20, 30], DEV)

    def step():
        a.append(k, v, None, table=tab, q=q, q_out=qo, q_norm=w, k_norm=w)
        # (their bits: NaN among the codes is not equal to itself)
        return [x.view(torch.int16) for x in m.kv_read_paged(cu, 30, **a.c, **a.where, **a.s)]

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    s = torch.cuda.Stream()
    for i in range(3):
        qkv.copy_(au.queries(2, 8, D, BF, 90 + i, DEV))
        a.where["last_page_len"].copy_(au.i32([5 + i, 14 + 2 * i], DEV))
        start = [x.clone() for x in (*a.c.values(), *a.s.values())]
        g.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in (qo, *out, *(y.view(torch.uint8) for y in a.c.values()), *a.s.values())]
        for x, y in zip((*a.c.values(), *a.s.values()), start):
            x.copy_(y)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            eager = step()
        s.synchronize()
        now = [qo, *eager, *(y.view(torch.uint8) for y in a.c.values()), *a.s.values()]
        assert all(torch.equal(x, y) for x, y in zip(kept, now))


def test_refusals():
    m = lib()
    a, H, D = Cache([20], 32, 16, 2, 64, 87), 2, 64
    kv = au.queries(3, 4, D, BF, 88, DEV)
    k, v = kv[:, :2], kv[:, 2:]
    cu = au.i32([0, 3], DEV)
    plain = dict(a.where, **{n: torch.zeros(x.shape, dtype=BF, device=DEV) for n, x in a.c.items()})
    for call, err in (
            (lambda: m.kv_append_paged(k, v, cu, **a.c, **a.where), ValueError),
            (lambda: m.kv_append_paged(k, v, cu, **a.c, **a.where, k_scale=a.s["k_scale"]), ValueError),
            (lambda: m.kv_append_paged(k, v, cu, **plain, **a.s), ValueError),
            (lambda: m.attention_prefill_paged(k, cu, **plain, **a.s), ValueError),
            (lambda: m.attention_prefill_paged(k, cu, **a.c, **a.where), ValueError),
            (lambda: m.attention_decode_paged(k[:1], **a.c, **a.where, **a.s, sinks=-1, window=3), m.GDNError),
            (lambda: m.kv_append_paged(k.float(), v.float(), cu, **a.c, **a.where, **a.s), m.GDNError),
            (lambda: m.kv_append_paged(k, v, cu, **a.c, **a.where, k_scale=a.s["k_scale"][:, :1], v_scale=a.s["v_scale"]), ValueError),
            (lambda: m.kv_append_paged(k, v, cu, a.c["k_cache"], plain["v_cache"], **a.where, **a.s), TypeError),
            (lambda: m.kv_read_paged(cu, 3, **plain, **a.s), TypeError),
            (lambda: m.kv_read_paged(cu, 3, **a.c, **a.where, **a.s, dtype=torch.int32), TypeError),
            (lambda: m.kv_read_paged(cu, -3, **a.c, **a.where, **a.s), m.GDNError),
            (lambda: m.kv_read_paged(cu, 3, **a.c, **a.where, **a.s, k_out=k[:, :1]), ValueError)):
        with pytest.raises(err):
            call()
