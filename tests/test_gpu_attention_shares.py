"""Attention where a workgroup's or a wave's share is long, crosses many sequences
or is one of many parts of a run: histories staged in several pieces on pages of
any size, stretches of empty sequences, joins of a few and of hundreds of parts."""

import math

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


def dense_of(q, k, v, past, softcap=0.0):
    """oracle.attention.softmax_rows's five arrays of one causal sequence, on the GPU in 64 bits, a head at a time."""
    T, H, D = q.shape
    G, L, scale = H // k.shape[1], k.shape[0], 1.0 / math.sqrt(D)
    hidden = torch.arange(L, device=DEV)[None, :] > past + torch.arange(T, device=DEV)[:, None]
    rows = [[], [], [], [], []]
    for h in range(H):
        a, b, c = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        x = scale * (a @ b.t().contiguous())
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        reach = x.masked_fill(hidden, 0.0).abs().amax(dim=1)
        x = x.masked_fill(hidden, -math.inf)
        p = torch.softmax(x, dim=1)
        spread = scale * (a.abs() @ b.abs().t().contiguous()).masked_fill(hidden, 0.0).amax(dim=1)
        for dst, y in zip(rows, (p @ c, torch.logsumexp(x, dim=1), p @ c.abs(), spread, reach)):
            dst.append(y)
    return [torch.stack(r, dim=1).cpu().numpy() for r in rows]


@pytest.mark.parametrize("D,dtype,page,cap", [(64, HF, 5, 0.0), (64, BF, 100, 20.0), (128, BF, 1, 0.0), (128, HF, 100, 0.0),
                                              (256, BF, 7, 0.0), (128, BF, 16, 0.0), (256, HF, 896, 10.0)])
def test_long_shares_on_any_page(D, dtype, page, cap):
    """More keys a share than places are staged at a time (2,048 of single rows), and every
    tile of a share but its last few unchecked."""
    new, past, Hk, G = 800, 7001, 2, 12
    L = new + past
    pages = -(-L // page)
    gen = torch.Generator(device=DEV).manual_seed(page + D)
    kv = torch.randn(2, pages * page, Hk, D, generator=gen, device=DEV).to(dtype)
    kv[:, L:] = math.nan
    ids = torch.randperm(pages, generator=gen, device=DEV)
    paged = torch.empty(2, pages, page, Hk, D, dtype=dtype, device=DEV)
    paged[:, ids] = kv.view(2, pages, page, Hk, D)
    q = torch.randn(new, Hk * G, D, generator=gen, device=DEV).to(dtype)
    o, lse = lib().attention_prefill_paged(q, au.i32([0, new], DEV), paged[0], paged[1], ids.to(torch.int32),
                                           au.i32([0, pages], DEV), page, au.i32([L - (pages - 1) * page], DEV),
                                           softcap=cap, return_lse=True)
    torch.cuda.synchronize()
    au.check_attention(o, lse, dense_of(q, kv[0, :L], kv[1, :L], past, cap), D, dtype, cap)


def check_decode(lens, page, Hk, G, D, dtype, seed, **kw):
    c = au.batch(lens, page, Hk, D, dtype, seed, DEV)
    q = au.queries(len(lens), Hk * G, D, dtype, seed + 1, DEV)
    o, lse = lib().attention_decode_paged(q, **c, return_lse=True, **kw)
    torch.cuda.synchronize()
    ref = oatt.attention_paged(au.f64(q), None, au.f64(c["k_cache"]), au.f64(c["v_cache"]), c["page_indices"].tolist(),
                               c["page_indptr"].tolist(), page, c["last_page_len"].tolist(), **kw)
    au.check_attention(o, lse, ref, D, dtype, kw.get("softcap", 0.0))


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (256, BF)])
def test_stretches_of_empty_sequences(D, dtype):
    """Runs of one wave more than 64 sequences apart, thousands of sequences of one or two tiles."""
    lens = ([1, 3, 40, 2] * 25 + [0] * 100) * 12 + [0] * 90 + [70]
    check_decode(lens, 4, 2, 2, D, dtype, D)


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, HF), (256, BF)])
@pytest.mark.parametrize("lens,G", [([9000, 3], 2), ([5000], 17), ([2000, 0, 1500, 33], 16)])
def test_few_runs_of_many_parts(D, dtype, lens, G):
    check_decode(lens, 32, 1, G, D, dtype, 5 + D)


@pytest.mark.parametrize("G", [1, 5, 20])
def test_many_runs_of_a_few_parts(G):
    check_decode([300, 1, 700, 0, 150] * 40, 16, 2 if G < 20 else 1, G, 128, BF, G, window=600)
