"""GPU parity of the rotary operators and the append against fp64: tables with
every scaling, both pair layouts, part of the head, types, strides, in place, the
gradient against the formula and against differences, and what the append may
and may not write."""

import numpy as np
import pytest
import torch

import attention_util as au
from oracle import attention as oatt

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def lib():
    import paged_recurrent_state_amd as m
    m.load()
    return m


def close(got, want, x, dtype, rot, tab, what=""):
    a, u = au.rotation_bounds(x, dtype, rot, tab)
    err = np.abs(au.f64(got) - want)
    lim = a * (1 + u) + u * np.abs(want) + au.TINY[dtype]
    assert (err <= lim).all(), f"{what}: {float((err / lim).max()):.2f} times its bound"


SCALINGS = [dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0),
            dict(scaling="base", factor=8.0), dict(scaling="bands", factor=8.0, original=64.0),
            dict(scaling="bands", factor=16.0, original=4096.0, low_turns=1.0, high_turns=32.0, magnitude=1.277)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("rot", [64, 128, 20])
def test_table(kw, rot):
    n = 300
    got = lib().rope_table(n, rot, **kw)
    torch.cuda.synchronize()
    want = oatt.table(n, rot, **kw)
    # one rounding to fp32 of values up to the magnitude (< 2), and the fp64 angle's own error (a few
    # 2^-53 of at most n)
    assert np.abs(au.f64(got) - want).max() <= 2.0 ** -24 + 1e-12


def test_table_at_far_positions():
    """2^20 positions: angles of a million radians keep every bit of fp32."""
    got = lib().rope_table(1 << 20, 8)
    torch.cuda.synchronize()
    want = oatt.table(1 << 20, 8)
    assert np.abs(au.f64(got) - want).max() <= 2.0 ** -25 + 1e-9


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 64), (128, 32), (256, 64), (80, 80), (80, 20), (96, 48), (5, 2), (7, 6)])
def test_rope(dtype, interleaved, D, rot):
    T, Hq, Hk = 37, 5, 2
    tab = lib().rope_table(200, rot)
    pos = torch.randint(0, 200, (T,), generator=torch.Generator().manual_seed(D), dtype=torch.int64)
    q, k = au.queries(T, Hq, D, dtype, 1, DEV, 3.0), au.queries(T, Hk, D, dtype, 2, DEV)
    for p in (pos.to(DEV), pos.to(torch.int32).to(DEV)):
        qo, ko = lib().rope(q, k, tab, p, interleaved=interleaved)
        torch.cuda.synchronize()
        for got, x in ((qo, q), (ko, k)):
            x = au.f64(x)
            want = oatt.rotate(x, au.f64(tab), pos.tolist(), interleaved)
            close(got, want, x, dtype, rot, au.f64(tab))
            assert np.array_equal(au.f64(got)[..., rot:], x[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 64), (80, 20)])
def test_gradient(interleaved, D, rot):
    """With y = R x and the loss <w, y>, the gradient is R^T w: against the formula, and against
    differences of the loss along single inputs (the map is linear, so a difference is exact up to
    fp32 rounding)."""
    T, H = 9, 3
    m = lib()
    tab = m.rope_table(64, rot, scaling="linear", factor=2.0, magnitude=1.25)
    pos = torch.arange(5, 5 + T, device=DEV) * 4
    x, w = au.queries(T, H, D, FP, 3, DEV), au.queries(T, H, D, FP, 4, DEV)
    dx, none = m.rope_backward(w, None, tab, pos, interleaved=interleaved)
    assert none is None
    want = oatt.rotate(au.f64(w), au.f64(tab), pos.tolist(), interleaved, transposed=True)
    close(dx, want, au.f64(w), FP, rot, au.f64(tab))
    y0 = m.rope(x, None, tab, pos, interleaved=interleaved)[0].double()
    r = np.random.default_rng(5)
    for _ in range(12):
        t, h, d = int(r.integers(T)), int(r.integers(H)), int(r.integers(D))
        x2 = x.clone()
        x2[t, h, d] += 1.0
        y = m.rope(x2, None, tab, pos, interleaved=interleaved)[0].double()
        diff = ((y - y0) * w.double()).sum().item() / (x2[t, h, d] - x[t, h, d]).item()
        # y rounds to 2^-22 of a few units in each of two places
        assert abs(diff - dx[t, h, d].item()) <= 2.0 ** -18 * (1 + abs(diff))


def test_rope_then_backward_returns_the_rows():
    m = lib()
    tab = m.rope_table(128, 128)
    pos = torch.arange(100, device=DEV)
    x = au.queries(100, 4, 128, FP, 6, DEV)
    y = m.rope(x, x, tab, pos)
    z = m.rope_backward(*y, tab, pos)
    for a in z:
        # two maps of norm 1 + 2^-24 and two sets of rounded products
        assert (a - x).abs().max().item() <= 2.0 ** -20 * x.abs().max().item()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rope_in_place_strided_and_unaligned(dtype):
    m = lib()
    T, Hq, Hk, D, rot = 33, 6, 2, 64, 32
    tab = m.rope_table(64, rot)
    pos = torch.arange(T, device=DEV, dtype=torch.int32)
    qkv = au.queries(T, Hq + 2 * Hk, D, dtype, 8, DEV)
    want = m.rope(qkv[:, :Hq].contiguous(), qkv[:, Hq:Hq + Hk].contiguous(), tab, pos)
    got = qkv.clone()
    q, k = got[:, :Hq], got[:, Hq:Hq + Hk]
    qo, ko = m.rope(q, k, tab, pos, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert qo.data_ptr() == q.data_ptr()
    assert torch.equal(got[:, :Hq], want[0]) and torch.equal(got[:, Hq:Hq + Hk], want[1])
    assert torch.equal(got[:, Hq + Hk:], qkv[:, Hq + Hk:])
    # rows that start at odd elements
    flat = torch.empty(T * Hq * D + 3, dtype=dtype, device=DEV)
    odd = flat[3:].view(T, Hq, D)
    odd.copy_(qkv[:, :Hq])
    got = m.rope(odd, None, tab, pos)[0]
    assert torch.equal(got, want[0])
    # heads apart, tokens inside
    ht = qkv[:, :Hq].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(m.rope(ht, None, tab, pos)[0], want[0])


def test_rope_position_outside_the_table_gives_nan():
    m = lib()
    tab = m.rope_table(10, 32)
    q = au.queries(4, 2, 64, BF, 9, DEV)
    o, _ = m.rope(q, None, tab, torch.tensor([0, 10, -1, 1 << 40], device=DEV))
    torch.cuda.synchronize()
    assert torch.isfinite(o[0]).all()
    assert torch.isnan(o[1:, :, :32]).all() and torch.equal(o[:, :, 32:], q[:, :, 32:])


def test_rope_no_tokens_and_one():
    m = lib()
    tab = m.rope_table(4, 64)
    e = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    o, k = m.rope(e, e, tab, torch.empty(0, dtype=torch.int64, device=DEV))
    assert o.shape == k.shape == (0, 2, 64)
    q = au.queries(1, 1, 64, BF, 10, DEV)
    o, _ = m.rope(q, None, tab, torch.zeros(1, dtype=torch.int64, device=DEV))
    assert torch.equal(o, q)  # position 0 turns nothing


# ------------------------------------------------------------------- append

def append_case(new, past, page, Hq, Hk, D, dtype, seed, heads_first=False):
    lens = [a + b for a, b in zip(new, past)]
    c = au.batch(lens, page, Hk, D, dtype, seed, DEV, heads_first=heads_first)
    T = sum(new)
    qkv = au.queries(T, Hq + 2 * Hk, D, dtype, seed + 1, DEV)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return c, qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], cu


def check_append(new, past, page, Hq, Hk, D, rot, dtype, seed, interleaved=False, heads_first=False, decode=False):
    m = lib()
    c, q, k, v, cu = append_case(new, past, page, Hq, Hk, D, dtype, seed, heads_first)
    before_k, before_v = c["k_cache"].clone(), c["v_cache"].clone()
    tab = m.rope_table(max(a + b for a, b in zip(new, past)), rot) if rot else None
    qo = m.kv_append_paged(k, v, None if decode else au.i32(cu, DEV), **c, table=tab, interleaved=interleaved, q=q)
    torch.cuda.synchronize()
    pos = [p + i for n, p in zip(new, past) for i in range(n)]
    tb = au.f64(tab) if rot else np.zeros((0, 0))
    turn = (lambda x: oatt.rotate(au.f64(x), tb, pos, interleaved)) if rot else au.f64
    close(qo, turn(q), au.f64(q), dtype, rot, tb, "q")
    want_k = turn(k)
    t = 0
    for b in range(len(new)):
        where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), page, b)
        for j in range(past[b], past[b] + new[b]):
            p, i = where[j]
            close(c["k_cache"][p, i][None], want_k[t][None], au.f64(k[t])[None], dtype, rot, tb, "k")
            assert torch.equal(c["v_cache"][p, i], v[t])
            before_k[p, i], before_v[p, i] = c["k_cache"][p, i], c["v_cache"][p, i]
            t += 1
    bits = torch.int32 if dtype == FP else torch.int16
    for a, b in ((before_k, c["k_cache"]), (before_v, c["v_cache"])):
        assert torch.equal(a.contiguous().view(bits), b.contiguous().view(bits)), "a slot that is not new changed"


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads_first", [False, True])
def test_append_types_and_layouts(dtype, interleaved, heads_first):
    check_append([20, 0, 1, 7], [3, 5, 31, 0], 16, 4, 2, 64, 32, dtype, 20, interleaved, heads_first)


@pytest.mark.parametrize("page", [1, 7, 64, 896])
@pytest.mark.parametrize("D,rot", [(128, 128), (256, 64), (128, 0), (80, 20)])
def test_append_pages_and_heads(page, D, rot):
    check_append([9, 30], [60, 0], page, 3, 1, D, rot, BF, 21)


def test_append_one_token_each():
    past = [0, 1, 15, 16, 17, 100, 63, 64]
    check_append([1] * 8, past, 16, 4, 2, 128, 64, BF, 22, decode=True)
    check_append([1] * 8, past, 16, 4, 2, 128, 64, BF, 22)


def test_append_many_sequences():
    new = [(i * 5) % 4 for i in range(200)]
    past = [(i * 3) % 40 for i in range(200)]
    check_append(new, past, 16, 2, 1, 64, 64, BF, 23)


def test_append_without_queries_and_with_strides():
    m = lib()
    c, q, k, v, cu = append_case([5, 3], [7, 0], 16, 4, 2, 64, BF, 24)
    tab = m.rope_table(64, 64)
    both = torch.stack([c["k_cache"], c["v_cache"]], dim=1)  # pages of keys and values in turn
    c2 = dict(c, k_cache=both[:, 0], v_cache=both[:, 1])
    assert m.kv_append_paged(k, v, au.i32(cu, DEV), **c, table=tab) is None
    assert m.kv_append_paged(k, v, au.i32(cu, DEV), **c2, table=tab) is None
    torch.cuda.synchronize()
    for n in ("k_cache", "v_cache"):
        assert torch.equal(c[n].view(torch.int16), c2[n].contiguous().view(torch.int16))


def test_append_more_tokens_than_the_table_holds_writes_none_of_the_excess():
    m = lib()
    c, q, k, v, cu = append_case([6], [0], 16, 2, 1, 64, BF, 25)
    c["last_page_len"] = au.i32([4], DEV)  # the sequence holds 4 tokens, 6 are new
    c["k_cache"].fill_(3.0)
    c["v_cache"].fill_(3.0)
    m.kv_append_paged(k, v, au.i32(cu, DEV), **c)
    torch.cuda.synchronize()
    p = int(c["page_indices"][0])
    assert torch.equal(c["k_cache"][p, :4], k[2:]) and torch.equal(c["v_cache"][p, :4], v[2:])
    rest = c["k_cache"].clone()
    rest[p, :4] = 3.0
    assert (rest == 3.0).all()


def test_append_page_past_32_bits():
    m = lib()
    pages, page, Hk, D = 36000, 64, 8, 128
    kv = torch.empty(2, pages, page, Hk, D, dtype=BF, device=DEV)
    k, v = au.queries(2, Hk, D, BF, 26, DEV), au.queries(2, Hk, D, BF, 27, DEV)
    m.kv_append_paged(k, v, None, kv[0], kv[1], au.i32([35999, 35000, 2], DEV), au.i32([0, 1, 3], DEV), page,
                      au.i32([64, 1], DEV))
    torch.cuda.synchronize()
    assert torch.equal(kv[0, 35999, 63], k[0]) and torch.equal(kv[1, 2, 0], v[1])


def test_append_graph_replays():
    m = lib()
    c, q, k, v, cu = append_case([1, 1], [40, 3], 16, 4, 2, 128, BF, 28)
    q, k, v = (x.clone() for x in (q, k, v))
    tab = m.rope_table(64, 128)
    qo = torch.empty_like(q)
    m.kv_append_paged(k, v, None, **c, table=tab, q=q, q_out=qo)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv_append_paged(k, v, None, **c, table=tab, q=q, q_out=qo)
    for step in range(3):
        q.copy_(au.queries(2, 4, 128, BF, 60 + step, DEV))
        k.copy_(au.queries(2, 2, 128, BF, 70 + step, DEV))
        c["last_page_len"].copy_(au.i32([10 + step, 4 + step], DEV))
        g.replay()
        torch.cuda.synchronize()
        got = qo.clone(), c["k_cache"].clone()
        m.kv_append_paged(k, v, None, **c, table=tab, q=q, q_out=qo)
        torch.cuda.synchronize()
        assert torch.equal(got[0], qo) and torch.equal(got[1].view(torch.int16), c["k_cache"].view(torch.int16))
