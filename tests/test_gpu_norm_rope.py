"""GPU parity of the norm of query and key heads with the rotation, of its gradient and
of the append that norms on the way, against fp64: types, head sizes and piece widths,
weights, strides, in place, positions outside the table, automatic differentiation,
large calls, other streams and graphs."""

import numpy as np
import pytest
import torch

import attention_util as au
from oracle import attention as oatt
from oracle import norms

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5

# A row's sum of squares: at most 16 fused steps a lane, six exchanges and the last one, each off by 2^-24 of it;
# the inverse root halves that and adds 2^-22, the products with it and the weight (a sum with the offset) 2^-22,
# the rotation 2^-22 of its pair: 2^-19 in all, relative to the row's largest value.
REL = 2.0 ** -19


def lib():
    import paged_recurrent_state_amd as m
    m.load()
    return m


def close(got, want, dtype, what="", rel=REL, of=None):
    of = np.abs(want).max(axis=-1, keepdims=True) * 2.0 if of is None else of
    u = au.UNIT[dtype]
    lim = of * rel * (1 + u) + u * np.abs(want) + au.TINY[dtype]
    err = np.abs(au.f64(got) - want)
    assert (err <= lim).all(), f"{what}: {float((err / lim).max()):.2f} times its bound"


def setup(T, Hq, Hk, D, rot, dtype, wide, seed=0, offset=0.0):
    q, k = au.queries(T, Hq, D, dtype, seed, DEV, 2.0), au.queries(T, Hk, D, dtype, seed + 1, DEV)
    gen = torch.Generator().manual_seed(seed + 2)
    wq, wk = ((1 - offset + 0.3 * torch.randn(D, generator=gen)).to(FP if wide else dtype).to(DEV) for _ in range(2))
    tab = lib().rope_table(50, rot)
    pos = torch.arange(T, device=DEV) * 7 % 50
    return q, k, wq, wk, tab, pos


def check_grad(got, g, x, w, tab, pos, offset, near, dtype, what):
    x, g, w64, tab = au.f64(x), au.f64(g), au.f64(w), au.f64(tab)
    dx, dw = norms.norm_rope_grad(g, x, w64, tab, pos.tolist(), EPS, offset, near)
    r = 1 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + EPS)
    y = oatt.rotate(g, tab, pos.tolist(), near, transposed=True)
    n = np.abs(y * (offset + w64))
    # the terms that cancel: each is off by REL of its row's largest
    of = r * (n.max(axis=-1, keepdims=True) * 2 + np.abs(x) * r * r * (n * np.abs(x)).mean(axis=-1, keepdims=True))
    close(got[0], dx, dtype, what, 4 * REL, of)
    # a sum over the rows in fp32, of at most 64 steps of 2^-24 of its terms at these sizes, each term off by 2 REL
    terms = (np.abs(y * x * r) + np.abs(y).max(axis=-1, keepdims=True) * np.abs(x) * r).sum(axis=(0, 1))
    lim = terms * (2.0 ** -18 + 2 * REL) + au.UNIT[w.dtype] * np.abs(dw) + au.TINY[w.dtype]
    assert (np.abs(au.f64(got[1]) - dw) <= lim).all(), what + " weight"


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("D,rot,wide,offset", [(64, 64, False, 0.0), (128, 64, True, 1.0), (128, 32, False, 1.0), (256, 64, True, 0.0),
                                               (80, 80, False, 0.0), (80, 20, True, 0.0), (96, 48, False, 1.0), (5, 2, False, 0.0),
                                               (7, 6, True, 1.0), (130, 6, False, 0.0), (512, 512, True, 0.0), (2, 2, False, 0.0),
                                               (509, 30, True, 0.0), (300, 4, False, 1.0)])
def test_forward_and_gradient(dtype, near, D, rot, wide, offset):
    T, Hq, Hk = 23, 5, 2
    m = lib()
    q, k, wq, wk, tab, pos = setup(T, Hq, Hk, D, rot, dtype, wide, D, offset)
    more = dict(eps=EPS, weight_offset=offset, interleaved=near)
    for p in (pos, pos.to(torch.int32)):
        out = m.norm_rope(q, k, wq, wk, tab, p, **more)
        torch.cuda.synchronize()
        for got, x, w in zip(out, (q, k), (wq, wk)):
            want = norms.norm_rope(au.f64(x), au.f64(w), au.f64(tab), pos.tolist(), EPS, offset, near)
            close(got, want, dtype)
    gq, gk = au.queries(T, Hq, D, dtype, 50, DEV), au.queries(T, Hk, D, dtype, 51, DEV)
    dq, dk, dwq, dwk = m.norm_rope_backward(gq, gk, q, k, wq, wk, tab, pos, **more)
    torch.cuda.synchronize()
    assert dwq.dtype == wq.dtype and dq.dtype == dtype
    check_grad((dq, dwq), gq, q, wq, tab, pos, offset, near, dtype, "q")
    check_grad((dk, dwk), gk, k, wk, tab, pos, offset, near, dtype, "k")
    alone = m.norm_rope_backward(gq, None, q, None, wq, None, tab, pos, **more)
    assert torch.equal(alone[0], dq) and alone[1] is None and alone[3] is None


def test_gradient_against_differences():
    m = lib()
    T, H, D, rot = 6, 3, 64, 32
    q, _, wq, _, tab, pos = setup(T, H, 1, D, rot, FP, True, 3)
    g = au.queries(T, H, D, FP, 4, DEV)
    dq, _, dw, _ = m.norm_rope_backward(g, None, q, None, wq, None, tab, pos, EPS)

    def loss(x, w):
        return (m.norm_rope(x, None, w, None, tab, pos, EPS)[0].double() * g.double()).sum().item()

    r = np.random.default_rng(5)
    h = 2.0 ** -7  # the loss is a sum of 1152 values off by 2^-20 at most; its third derivative is of order one
    for _ in range(10):
        t, i, d = int(r.integers(T)), int(r.integers(H)), int(r.integers(D))
        e = torch.zeros_like(q)
        e[t, i, d] = h
        diff = (loss(q + e, wq) - loss(q - e, wq)) / ((q + e)[t, i, d] - (q - e)[t, i, d]).item()
        assert abs(diff - dq[t, i, d].item()) < 64 * 2.0 ** -20 / h + 16 * h * h
        e = torch.zeros_like(wq)
        e[d] = h
        diff = (loss(q, wq + e) - loss(q, wq - e)) / ((wq + e)[d] - (wq - e)[d]).item()
        assert abs(diff - dw[d].item()) < 64 * 2.0 ** -20 / h


@pytest.mark.parametrize("dtype", [BF, FP])
def test_views_in_place_and_unaligned(dtype):
    m = lib()
    T, Hq, Hk, D, rot = 33, 6, 2, 64, 32
    tab, pos = m.rope_table(64, rot), torch.arange(T, device=DEV, dtype=torch.int32)
    qkv = au.queries(T, Hq + 2 * Hk, D, dtype, 8, DEV)
    wq, wk = torch.rand(D, device=DEV) + 0.5, torch.rand(D, device=DEV) + 0.5
    want = m.norm_rope(qkv[:, :Hq].contiguous(), qkv[:, Hq:Hq + Hk].contiguous(), wq, wk, tab, pos)
    got = qkv.clone()
    q, k = got[:, :Hq], got[:, Hq:Hq + Hk]
    a, b = m.norm_rope(q, k, wq, wk, tab, pos, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert a.data_ptr() == q.data_ptr() and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(got[:, Hq + Hk:], qkv[:, Hq + Hk:])
    ht = qkv[:, :Hq].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(m.norm_rope(ht, None, wq, None, tab, pos)[0], want[0])
    flat = torch.empty(T * Hq * D + 3, dtype=dtype, device=DEV)
    odd = flat[3:].view(T, Hq, D)
    odd.copy_(qkv[:, :Hq])
    pad = torch.empty(D + 1, device=DEV)
    pad[1:] = wq
    got = m.norm_rope(odd, None, pad[1:], None, tab, pos)[0]
    ref = norms.norm_rope(au.f64(odd), au.f64(wq), au.f64(tab), pos.tolist(), 1e-6)
    close(got, ref, dtype)
    gq = au.queries(T, Hq, D, dtype, 9, DEV)
    dq = m.norm_rope_backward(gq, None, qkv[:, :Hq], None, wq, None, tab, pos)
    odd_dq = m.norm_rope_backward(gq, None, odd, None, wq, None, tab, pos)
    check_grad((odd_dq[0], odd_dq[2]), gq, odd, wq, tab, pos, 0.0, False, dtype, "odd")
    check_grad((dq[0], dq[2]), gq, qkv[:, :Hq], wq, tab, pos, 0.0, False, dtype, "view")


def test_rows_of_zeros_infinities_and_far_positions():
    m = lib()
    D = 64
    tab = m.rope_table(10, 32)
    w = torch.ones(D, dtype=BF, device=DEV)
    x = au.queries(6, 1, D, BF, 9, DEV)
    x[0] = 0
    x[1, 0, 5] = float("inf")
    x[2, 0, 40] = float("nan")
    pos = torch.tensor([1, 2, 3, 10, -1, 4], device=DEV)
    o = m.norm_rope(x, None, w, None, tab, pos)[0]
    torch.cuda.synchronize()
    assert (o[0] == 0).all()
    assert torch.isnan(o[1, 0, 5]) and torch.isnan(o[2]).all()
    assert torch.isnan(o[3:5, :, :32]).all() and torch.isfinite(o[3:5, :, 32:]).all() and torch.isfinite(o[5]).all()
    # eps 0 and a row of zeros: 0 / 0, as the formula has it
    assert torch.isnan(m.norm_rope(x[:1], None, w, None, tab, pos[:1], eps=0.0)[0]).all()


@pytest.mark.parametrize("T", [0, 1, 2])
def test_few_tokens(T):
    m = lib()
    q, k, wq, wk, tab, pos = setup(T, 3, 1, 128, 128, BF, False, 11)
    a, b = m.norm_rope(q, k, wq, wk, tab, pos, EPS)
    assert a.shape == q.shape and b.shape == k.shape
    g = torch.ones_like(q)
    dq, dk, dwq, dwk = m.norm_rope_backward(g, torch.ones_like(k), q, k, wq, wk, tab, pos, EPS)
    torch.cuda.synchronize()
    if T == 0:
        assert (dwq == 0).all() and (dwk == 0).all()
    else:
        check_grad((dq, dwq), g, q, wq, tab, pos, 0.0, False, BF, "q")


def test_no_heads():
    m = lib()
    q, k, wq, wk, tab, pos = setup(4, 2, 1, 64, 64, BF, False, 12)
    none = q[:, :0]
    a, b = m.norm_rope(none, k, wq, wk, tab, pos)
    assert a.shape == (4, 0, 64) and torch.equal(b, m.norm_rope(k, None, wk, None, tab, pos)[0])
    dq, dk, dwq, dwk = m.norm_rope_backward(none, k, none, k, wq, wk, tab, pos)
    assert (dwq == 0).all() and torch.equal(dwk, m.norm_rope_backward(k, None, k, None, wk, None, tab, pos)[2])


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_large_calls_pass_the_caches(near, dtype):
    """Over 32 MiB: checked at rows spread over the call, the weights' gradient against torch's in 64 bits."""
    m = lib()
    T, Hq, Hk, D = 9001, 16, 4, 128
    q, k, wq, wk, _, _ = setup(T, Hq, Hk, D, 64, dtype, True, 13)
    tab, pos = m.rope_table(T, 64), torch.arange(T, device=DEV)
    a, b = m.norm_rope(q, k, wq, wk, tab, pos, EPS, 0.0, near)
    gq, gk = au.queries(T, Hq, D, dtype, 14, DEV), au.queries(T, Hk, D, dtype, 15, DEV)
    dq, dk, dwq, dwk = m.norm_rope_backward(gq, gk, q, k, wq, wk, tab, pos, EPS, 0.0, near)
    again = m.norm_rope_backward(gq, gk, q, k, wq, wk, tab, pos, EPS, 0.0, near)
    torch.cuda.synchronize()
    for x, y in zip((dq, dk, dwq, dwk), again):
        assert torch.equal(x, y), "the sums' order is not fixed"
    at = torch.arange(0, T, 613, device=DEV)
    for out, grad, g, x, w in ((a, dq, gq, q, wq), (b, dk, gk, k, wk)):
        close(out[at], norms.norm_rope(au.f64(x[at]), au.f64(w), au.f64(tab), at.tolist(), EPS, 0.0, near), dtype)
        dx, _ = norms.norm_rope_grad(au.f64(g[at]), au.f64(x[at]), au.f64(w), au.f64(tab), at.tolist(), EPS, 0.0, near)
        close(grad[at], dx, dtype, rel=16 * REL)
    for dw, g, x in ((dwq, gq, q), (dwk, gk, k)):
        y = m.rope_backward(g.float(), None, tab, pos, near)[0].double()
        xr = x.double() * (x.double().square().mean(-1, keepdim=True) + EPS).rsqrt()
        want, terms = (y * xr).sum((0, 1)), (y * xr).abs().sum((0, 1))
        # partial sums of at most 64 rows, then of some hundred workgroups a lane, then six steps
        assert ((dw.double() - want).abs() <= terms * 2.0 ** -16).all()


def test_automatic_differentiation():
    m = lib()
    T, Hq, Hk, D = 9, 4, 2, 64
    qkv = au.queries(T, Hq + 2 * Hk, D, FP, 16, DEV).requires_grad_()
    wq, wk = (torch.rand(D, device=DEV) + 0.5).requires_grad_(), (torch.rand(D, device=DEV) + 0.5).requires_grad_()
    tab, pos = m.rope_table(40, 32), torch.arange(T, device=DEV)
    q, k, _ = qkv.split([Hq, Hk, Hk], dim=1)
    a, b = m.norm_rope(q, k, wq, wk, tab, pos, EPS)
    ga, gb = torch.randn_like(a), torch.randn_like(b)
    torch.autograd.backward([a, b], [ga, gb])
    dq, dk, dwq, dwk = m.norm_rope_backward(ga, gb, q.detach(), k.detach(), wq.detach(), wk.detach(), tab, pos, EPS)
    assert torch.equal(qkv.grad[:, :Hq], dq) and torch.equal(qkv.grad[:, Hq:Hq + Hk], dk)
    assert (qkv.grad[:, Hq + Hk:] == 0).all() and torch.equal(wq.grad, dwq) and torch.equal(wk.grad, dwk)
    # one output alone, and a broadcast gradient
    for t in (qkv, wq, wk):
        t.grad = None
    q, k, _ = qkv.split([Hq, Hk, Hk], dim=1)
    m.norm_rope(q, k, wq, wk, tab, pos, EPS)[1].sum().backward()
    ones = torch.ones_like(gb)
    want = m.norm_rope_backward(ones, None, k.detach(), None, wk.detach(), None, tab, pos, EPS)
    assert torch.equal(qkv.grad[:, Hq:Hq + Hk], want[0]) and torch.equal(wk.grad, want[2])
    assert wq.grad is None and (qkv.grad[:, :Hq] == 0).all()
    # what is refused
    with pytest.raises(RuntimeError, match="q_out"):
        m.norm_rope(q, None, wq, None, tab, pos, q_out=torch.empty_like(q))
    with pytest.raises(RuntimeError, match="table"):
        m.norm_rope(q, None, wq, None, tab.clone().requires_grad_(), pos)
    y = m.norm_rope(q, None, wq, None, tab, pos, EPS)[0]
    g, = torch.autograd.grad(y.square().sum(), wq, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    with torch.no_grad():
        assert not m.norm_rope(q, None, wq, None, tab, pos)[0].requires_grad


def test_refusals():
    m = lib()
    q, k, wq, wk, tab, pos = setup(4, 2, 1, 64, 64, BF, False, 17)
    for call, err in (
            (lambda: m.norm_rope(q, k, wq, None, tab, pos), ValueError),
            (lambda: m.norm_rope(q, k, None, wk, tab, pos), ValueError),
            (lambda: m.norm_rope(q, k, wq, wk.float(), tab, pos), TypeError),
            (lambda: m.norm_rope(q, k, wq.half(), wk.half(), tab, pos), TypeError),
            (lambda: m.norm_rope(q, k, wq[:32], wk, tab, pos), ValueError),
            (lambda: m.norm_rope(q, k, wq, wk, tab, pos[:3]), ValueError),
            (lambda: m.norm_rope(q, k, wq, wk, tab, pos.float()), TypeError),
            (lambda: m.norm_rope(q, k, wq, wk, tab, pos, eps=-1.0), m.GDNError),
            (lambda: m.norm_rope_backward(q, k, q, None, wq, None, tab, pos), ValueError),
            (lambda: m.norm_rope_backward(q, None, q, None, None, None, tab, pos), ValueError),
            (lambda: m.norm_rope_backward(q[:3], k, q, k, wq, wk, tab, pos), ValueError),
            (lambda: m.norm_rope_backward(q.half(), k, q, k, wq, wk, tab, pos), TypeError),
            (lambda: m.norm_rope_backward(q, k, q, k, wq, wk, tab, pos, workspace=torch.empty(8, device=DEV)), ValueError)):
        with pytest.raises(err):
            call()


def test_other_stream_and_graph():
    m = lib()
    q, k, wq, wk, tab, pos = setup(300, 4, 2, 128, 64, BF, True, 18)
    gq, gk = au.queries(300, 4, 128, BF, 19, DEV), au.queries(300, 2, 128, BF, 20, DEV)

    def both():
        return (*m.norm_rope(q, k, wq, wk, tab, pos), *m.norm_rope_backward(gq, gk, q, k, wq, wk, tab, pos))

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for step in range(3):
        q.copy_(au.queries(300, 4, 128, BF, 30 + step, DEV))
        gk.copy_(au.queries(300, 2, 128, BF, 40 + step, DEV))
        g.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, both()))


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,rot,which", [(64, 32, "qk"), (128, 128, "q"), (128, 0, "qk"), (256, 64, "k"), (80, 20, "qk")])
def test_append_norms_on_the_way(dtype, D, rot, which):
    m = lib()
    new, past, Hq, Hk, page = [9, 0, 1, 20], [3, 5, 31, 0], 4, 2, 16
    c = au.batch([a + b for a, b in zip(new, past)], page, Hk, D, dtype, 21, DEV)
    qkv = au.queries(30, Hq + 2 * Hk, D, dtype, 22, DEV)
    q, k, v = qkv.split([Hq, Hk, Hk], dim=1)
    wq, wk = torch.rand(D, device=DEV).to(dtype) + 0.5, torch.rand(D, device=DEV).to(dtype) + 0.5
    tab = m.rope_table(64, rot) if rot else None
    pos = [p + i for n, p in zip(new, past) for i in range(n)]
    kw = dict(q_norm=wq if "q" in which else None, k_norm=wk if "k" in which else None, eps=EPS, norm_offset=0.5)
    before = c["k_cache"].clone()
    cu = au.i32([0, 9, 9, 10, 30], DEV)
    qo = m.kv_append_paged(k, v, cu, **c, table=tab, q=q, **kw)
    torch.cuda.synchronize()
    tb = au.f64(tab) if rot else np.zeros((64, 0))

    def want(x, w, on):
        return norms.norm_rope(au.f64(x), au.f64(w), tb, pos, EPS, 0.5) if on else oatt.rotate(au.f64(x), tb, pos)

    close(qo, want(q, wq, "q" in which), dtype, "q")
    wk_ = want(k, wk, "k" in which)
    t = 0
    for b in range(4):
        where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), page, b)
        for j in range(past[b], past[b] + new[b]):
            p, i = where[j]
            close(c["k_cache"][p, i][None], wk_[t][None], dtype, "k")
            assert torch.equal(c["v_cache"][p, i], v[t])
            before[p, i] = c["k_cache"][p, i]
            t += 1
    bits = torch.int32 if dtype == FP else torch.int16
    assert torch.equal(before.view(bits), c["k_cache"].view(bits)), "a slot that is not new changed"
    with pytest.raises(ValueError, match="q_norm"):
        m.kv_append_paged(k, v, cu, **c, table=tab, q_norm=wq)
