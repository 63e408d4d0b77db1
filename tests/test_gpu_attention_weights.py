"""Weights far below a row's largest: one heavy key whose values are zero beside tens
of thousands of light keys that hold all the output, and scores that rise through
the whole range of the element type."""

import math

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


def dense(q, k, v):
    """softmax_rows's five arrays of rows q [R, D] that see all of k, v [L, D], in 64 bits."""
    scale = 1.0 / math.sqrt(q.shape[1])
    q, k, v = q.double(), k.double().t().contiguous(), v.double()
    rows = [[], [], [], [], []]
    for lo in range(0, q.shape[0], 128):
        x = scale * (q[lo:lo + 128] @ k)
        p = torch.softmax(x, dim=1)
        spread = scale * (q[lo:lo + 128].abs() @ k.abs()).amax(dim=1)
        for dst, y in zip(rows, (p @ v, torch.logsumexp(x, dim=1), p @ v.abs(), spread, x.abs().amax(dim=1))):
            dst.append(y)
    return [torch.cat(r).cpu().numpy() for r in rows]


def long_bounds(ref, v, dim, dtype):
    """attention_bounds, and what it leaves out over many keys.

    Sums: L / 16 additions one after the other, of weights and of products, each rounded in fp32.
    Weights in fp16 have a least step of 2^-24, so that one is off by up to 2^-25 however small;
    the reference lies 2^7 under the row's largest or lower, so the weights sum to 2^7 at least
    and each value is off by up to 2^-32 of the quotient."""
    eo, el = au.attention_bounds(ref, dim, dtype)
    L = v.shape[0]
    eo = eo + 2 * (L / 16) * 2.0 ** -24 * ref[2]
    if dtype == HF:
        eo = eo + 2.0 ** -32 * v.double().abs().sum(dim=0).cpu().numpy()
    return eo, el + (L / 16) * 2.0 ** -24


def sink_case(L, D, dtype, p, spread, seed):
    """k, v [L, D] and 512 rows q: key 0 has probability p, whichever the row, and zero values; the
    others' scores are spread by `spread` and their values lie around 1."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(512, D, generator=gen, device=DEV)
    k = torch.randn(L, D, generator=gen, device=DEV) * spread
    v = 1.0 + 0.3 * torch.randn(L, D, generator=gen, device=DEV)
    q[:, 0], k[:, 0], v[0] = 8.0, 0.0, 0.0
    k[0] = 0.0
    k[0, 0] = (math.log(L * p / (1 - p)) + spread ** 2 / 2) * math.sqrt(D) / 8.0
    return q.to(dtype), k.to(dtype), v.to(dtype)


def pages_of(k, v, page, seqs):
    """One history, in permuted pages, that every one of `seqs` sequences has."""
    L, D = k.shape
    n = L // page
    ids = torch.randperm(n, generator=torch.Generator().manual_seed(n)).to(DEV)
    kv = torch.empty(2, n, page, 1, D, dtype=k.dtype, device=DEV)
    kv[0, ids], kv[1, ids] = k.view(n, page, 1, D), v.view(n, page, 1, D)
    return dict(k_cache=kv[0], v_cache=kv[1], page_indices=ids.to(torch.int32).repeat(seqs),
                page_indptr=au.i32([n * b for b in range(seqs + 1)], DEV), page_size=page,
                last_page_len=au.i32([page] * seqs, DEV))


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L,p,spread", [(32768, 0.9, 1.0), (131072, 0.9, 1.0), (131072, 0.95, 0.0), (131072, 0.98, 1.0),
                                        (131072, 0.98, 0.0), (32768, 0.98, 2.0)])
def test_heavy_first_key_without_values(D, dtype, L, p, spread):
    """256 sequences of one new token: as many runs as workgroups, none of them cut."""
    q, k, v = sink_case(L, D, dtype, p, spread, D + int(100 * p))
    c = pages_of(k, v, 64, 256)
    o, lse = lib().attention_prefill_paged(q.view(256, 2, D), au.i32(list(range(257)), DEV), **c, return_lse=True)
    torch.cuda.synchronize()
    ref = dense(q, k, v)
    eo, el = long_bounds(ref, v, D, dtype)
    worst = (np.abs(au.f64(o).reshape(512, D) - ref[0]) / eo).max()
    assert worst <= 1.0, f"output error {worst:.2f} times its bound"
    assert (np.abs(au.f64(lse).reshape(512) - ref[1]) <= el).all()


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_heavy_first_key_beside_a_value_that_is_not_finite(D, dtype):
    """A NaN in one column, so that every run is computed again with a following reference."""
    q, k, v = sink_case(32768, D, dtype, 0.98, 0.0, D)
    v[20000, 5] = math.nan
    c = pages_of(k, v, 64, 256)
    o = lib().attention_prefill_paged(q.view(256, 2, D), au.i32(list(range(257)), DEV), **c)
    torch.cuda.synchronize()
    assert torch.isnan(o[..., 5]).all()
    v[20000, 5] = 1.0
    ref = dense(q, k, v)
    eo, _ = long_bounds(ref, v, D, dtype)
    keep = [d for d in range(D) if d != 5]
    assert (np.abs(au.f64(o).reshape(512, D) - ref[0])[:, keep] <= eo[:, keep]).all()


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 5), (128, 64), (256, 16)])
@pytest.mark.parametrize("window,cap", [(0, 0.0), (300, 0.0), (0, 40.0)])
def test_scores_that_rise_through_the_range(D, page, dtype, window, cap):
    """Scores that rise by 0.06 a key over 1,500 keys (90, or up to the cap), other rows by less: references
    move again and again, at other keys in every row."""
    new, past, Hk, G = 100, 1400, 1, 2
    c = au.batch([new + past], page, Hk, D, dtype, 7, DEV)
    q = au.queries(new, Hk * G, D, dtype, 8, DEV, 0.5)
    where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), page, 0)
    q[..., 0] = 4.0 * torch.linspace(0.2, 1.0, new * G, device=DEV).view(new, G).to(dtype)
    for j, (p, i) in enumerate(where):
        c["k_cache"][p, i, 0, 0] = 0.06 * j * math.sqrt(D) / 4.0
    o, lse = lib().attention_prefill_paged(q, au.i32([0, new], DEV), **c, window=window, softcap=cap, return_lse=True)
    torch.cuda.synchronize()
    ref = oatt.attention_paged(au.f64(q), [0, new], au.f64(c["k_cache"]), au.f64(c["v_cache"]),
                               c["page_indices"].tolist(), c["page_indptr"].tolist(), page, c["last_page_len"].tolist(),
                               window=window, softcap=cap)
    au.check_attention(o, lse, ref, D, dtype, cap)
