"""Infinities and NaN among the values a row sees, at keys of the smallest weight: they
reach the row as themselves, however far below its largest score their keys lie,
before it or after it, inside a run and across its parts."""

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


def case(length, new, peaks, D, dtype, page, seed):
    """One sequence whose rows give each key of ``peaks`` {key: score} that score, and other keys small ones."""
    c = au.batch([length], page, 1, D, dtype, seed, DEV, gain=0.5)
    q = au.queries(new, 3, D, dtype, seed + 1, DEV, 0.5)
    q[..., 0] = 4.0
    where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), page, 0)
    for j, (p, i) in enumerate(where):
        if j in peaks:
            c["k_cache"][p, i] = 0.0
        c["k_cache"][p, i, 0, 0] = peaks.get(j, 0.0) * math.sqrt(D) / 4.0
    return q, c, where


def check(call, q, cu, c, where, odd, D, dtype, **kw):
    """``odd``: (key, column, value).  The columns without one keep to the oracle's values."""
    ref = oatt.attention_paged(au.f64(q), cu, au.f64(c["k_cache"]), au.f64(c["v_cache"]), c["page_indices"].tolist(),
                               c["page_indptr"].tolist(), c["page_size"], c["last_page_len"].tolist(), **kw)
    want = {}
    for key, col, x in odd:
        p, i = where[key]
        c["v_cache"][p, i, 0, col] = x
        want[col] = want.get(col, 0.0) + x
    o, lse = call(q, c)
    torch.cuda.synchronize()
    got = au.f64(o)
    for col, x in want.items():
        same = np.isnan(got[..., col]) if math.isnan(x) else got[..., col] == x
        assert same.all(), f"column {col}: {got[..., col].ravel()[:4]}, expected {x}"
    keep = [d for d in range(D) if d not in want]
    eo, el = au.attention_bounds(ref, D, dtype)
    assert (np.abs(got - ref[0])[..., keep] <= eo[..., keep]).all()
    assert (np.abs(au.f64(lse) - ref[1]) <= el).all()


def decode(q, c):
    return lib().attention_decode_paged(q, **c, return_lse=True)


def chunk(q, c):
    return lib().attention_prefill_paged(q, au.i32([0, q.shape[0]], DEV), **c, return_lse=True)


INF, NAN = math.inf, math.nan
ODD = [(7, 3, INF), (8, 9, -INF), (9, 20, NAN), (40, 30, INF), (60, 30, -INF), (150, 0, -INF), (151, 63, INF)]


@pytest.mark.parametrize("D,dtype", [(64, HF), (64, BF), (128, HF), (128, BF), (256, HF), (256, BF)])
@pytest.mark.parametrize("height", [2.0, 25.0, 40.0, 120.0, 300.0])
@pytest.mark.parametrize("peak", [0, 100, 299])
def test_far_below_the_largest_score(D, dtype, height, peak):
    q, c, where = case(300, 1, {peak: height}, D, dtype, 16, peak)
    check(decode, q, None, c, where, ODD, D, dtype)
    q, c, where = case(300, 1, {peak: height}, D, dtype, 16, peak)
    check(chunk, q, [0, 1], c, where, ODD, D, dtype)


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (128, HF), (256, BF)])
@pytest.mark.parametrize("peaks", [{10: 150.0}, {8900: 150.0}, {10: 60.0, 4000: 170.0, 8900: 290.0}])
def test_across_the_parts_of_a_run(D, dtype, peaks):
    odd = [(5, 3, INF), (3000, 9, -INF), (6000, 20, NAN), (8, 30, INF), (8950, 30, -INF), (8800, 0, -INF), (100, 63, INF)]
    q, c, where = case(9000, 1, peaks, D, dtype, 32, 3)
    check(decode, q, None, c, where, odd, D, dtype)
    q, c, where = case(9000, 1, peaks, D, dtype, 32, 3)
    check(chunk, q, [0, 1], c, where, odd, D, dtype)


@pytest.mark.parametrize("dtype", [HF, BF])
def test_sequences_beside_one_with_infinities(dtype):
    """The runs before and after one that is computed again, in the same wave's share."""
    lens = [5, 40, 33, 200, 64, 1, 90] * 200
    D, page = 128, 8
    c = au.batch(lens, page, 1, D, dtype, 5, DEV)
    q = au.queries(len(lens), 2, D, dtype, 6, DEV)
    odd = [b for b in range(len(lens)) if b % 5 == 2]
    ptr = c["page_indptr"].tolist()
    ref = oatt.attention_paged(au.f64(q), None, au.f64(c["k_cache"]), au.f64(c["v_cache"]), c["page_indices"].tolist(),
                               ptr, page, c["last_page_len"].tolist())
    for b in odd:
        c["v_cache"][c["page_indices"][ptr[b]], 0, 0, 7] = -INF
    o, lse = lib().attention_decode_paged(q, **c, return_lse=True)
    torch.cuda.synchronize()
    x = au.f64(o)
    assert np.isneginf(x[odd, :, 7]).all()
    x[odd, :, 7] = ref[0][odd, :, 7]
    eo, el = au.attention_bounds(ref, D, dtype)
    assert (np.abs(x - ref[0]) <= eo).all() and (np.abs(au.f64(lse) - ref[1]) <= el).all()
