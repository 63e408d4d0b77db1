"""Rows that see tokens but give none of them a weight: scores that are all -inf, in
runs that stay whole and in runs that are cut and joined."""

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


def batch_of(lens, new, page, D, dtype, keep):
    """Every key scores -inf but those at the positions ``keep`` of every sequence."""
    c = au.batch(lens, page, 1, D, dtype, D, DEV)
    q = au.queries(sum(new), 2, D, dtype, D + 1, DEV)
    q[..., 0] = 2.0
    for b in range(len(lens)):
        where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), page, b)
        for j, (p, i) in enumerate(where):
            c["k_cache"][p, i, 0, 0] = 0.5 if j in keep else -math.inf
    return q, c


def check(o, lse, q, cu, c, D, dtype, softcap=0.0):
    """The oracle's values with -inf scores made finite (2^16 lower than any other: a weight of 0), and NaN
    where nothing else is seen; a capped score of -inf is -softcap."""
    k = au.f64(c["k_cache"])
    far = np.isneginf(k)
    k[far] = -8192.0 * math.sqrt(D)
    if softcap:
        k[far] = -1e9
    ref = list(oatt.attention_paged(au.f64(q), cu, k, au.f64(c["v_cache"]), c["page_indices"].tolist(),
                                    c["page_indptr"].tolist(), c["page_size"], c["last_page_len"].tolist(), softcap=softcap))
    nothing = ~np.isneginf(ref[1]) & (ref[1] < -4096.0)
    # (the bounds' score terms are those of the keys that have a weight)
    ref[3], ref[4] = np.full_like(ref[3], 64.0), np.full_like(ref[4], 64.0)
    x, y = au.f64(o), au.f64(lse)
    assert np.isnan(x[nothing]).all() and np.isneginf(y[nothing]).all()
    eo, el = au.attention_bounds(ref, D, dtype, softcap)
    rest = ~nothing
    assert (np.abs(x - ref[0])[rest] <= eo[rest]).all()
    seen = rest & ~np.isneginf(ref[1])
    assert (np.isneginf(y) == (nothing | np.isneginf(ref[1]))).all()
    assert (np.abs(y[seen] - ref[1][seen]) <= el[seen]).all()
    return int(nothing.sum())


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (128, HF), (256, BF)])
@pytest.mark.parametrize("new,past", [([30], [20]), ([17], [5000]), ([40, 3, 1], [0, 2000, 300])])
def test_chunks(D, dtype, new, past):
    lens = [a + b for a, b in zip(new, past)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    for keep in (set(), {past[0] + new[0] // 2}, {0}):
        q, c = batch_of(lens, new, 16, D, dtype, keep)
        o, lse = lib().attention_prefill_paged(q, au.i32(cu, DEV), **c, return_lse=True)
        torch.cuda.synchronize()
        n = check(o, lse, q, cu, c, D, dtype)
        assert n == q.shape[0] * 2 if not keep else n < q.shape[0] * 2


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (256, HF)])
@pytest.mark.parametrize("lens", [[20], [5000], [1, 0, 300, 9000]])
def test_single_tokens(D, dtype, lens):
    for keep in (set(), {0}, {4000}):
        q, c = batch_of(lens, [1] * len(lens), 16, D, dtype, keep)
        o, lse = lib().attention_decode_paged(q, **c, return_lse=True)
        torch.cuda.synchronize()
        check(o, lse, q, None, c, D, dtype)


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF)])
def test_capped(D, dtype):
    for new, past in ((20, 30), (17, 4000)):
        q, c = batch_of([new + past], [new], 16, D, dtype, {3})
        o, lse = lib().attention_prefill_paged(q, au.i32([0, new], DEV), **c, softcap=2.0, return_lse=True)
        torch.cuda.synchronize()
        check(o, lse, q, [0, new], c, D, dtype, softcap=2.0)


def test_rows_that_see_no_token_in_runs_that_are_joined():
    """More new tokens than the sequence holds: the first of them lie before its start and see nothing."""
    D, page, held, new = 128, 16, 3000, 3040
    c = au.batch([held], page, 1, D, BF, 9, DEV)
    q = au.queries(new, 2, D, BF, 10, DEV)
    o, lse = lib().attention_prefill_paged(q, au.i32([0, new], DEV), **c, return_lse=True)
    torch.cuda.synchronize()
    assert (o[:40] == 0).all() and torch.isneginf(lse[:40]).all()
    ref = oatt.attention_paged(au.f64(q[40:]), [0, held], au.f64(c["k_cache"]), au.f64(c["v_cache"]),
                               c["page_indices"].tolist(), c["page_indptr"].tolist(), page, c["last_page_len"].tolist())
    au.check_attention(o[40:], lse[40:], ref, D, BF)
