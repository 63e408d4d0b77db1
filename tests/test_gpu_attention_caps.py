"""Capped scores over the whole range of caps: from ones that every score runs into
to ones so high that the tanh leaves the scores as they are."""

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


def check(got, q, cu, c, D, dtype, cap, short, **kw):
    ref = list(oatt.attention_paged(au.f64(q), cu, au.f64(c["k_cache"]), au.f64(c["v_cache"]), c["page_indices"].tolist(),
                                    c["page_indptr"].tolist(), c["page_size"], c["last_page_len"].tolist(), softcap=cap, **kw))
    if not short:
        # 2^-19 of the largest score, where attention_bounds has 2^-21 of it and of the cap
        ref[4] = 4 * ref[4]
        cap = 0.0
    au.check_attention(*got, ref, D, dtype, cap)


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (128, HF), (256, BF)])
@pytest.mark.parametrize("cap", [0.5, 5.0, 30.0, 64.0, 65.0, 1e3, 1e4, 1e6, 1e20, 1e30, 3e38])
@pytest.mark.parametrize("page,window", [(16, 0), (7, 0), (16, 200)])
def test_chunks(D, dtype, cap, page, window):
    new, past, Hk, G = [50, 3], [400, 700], 1, 3
    c = au.batch([a + b for a, b in zip(new, past)], page, Hk, D, dtype, D, DEV)
    q = au.queries(53, Hk * G, D, dtype, D + 1, DEV, 4.0)
    got = lib().attention_prefill_paged(q, au.i32([0, 50, 53], DEV), **c, softcap=cap, window=window, return_lse=True)
    torch.cuda.synchronize()
    check(got, q, [0, 50, 53], c, D, dtype, cap, cap <= 64, window=window)


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (128, HF), (256, BF)])
@pytest.mark.parametrize("cap", [0.5, 5.0, 30.0, 64.0, 65.0, 1e3, 1e4, 1e6, 1e20, 1e30, 3e38])
def test_single_tokens(D, dtype, cap):
    lens = [1, 33, 900, 0, 4000]
    c = au.batch(lens, 16, 1, D, dtype, D + 2, DEV)
    q = au.queries(len(lens), 3, D, dtype, D + 3, DEV, 4.0)
    got = lib().attention_decode_paged(q, **c, softcap=cap, return_lse=True)
    torch.cuda.synchronize()
    check(got, q, None, c, D, dtype, cap, False)


@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("cap", [40.0, 100.0])
def test_scores_around_the_quarter_of_the_cap(dtype, cap):
    """Two keys whose scores straddle the place where the one form takes over from the other, and their
    difference in the log-sum-exp."""
    D = 64
    c = au.batch([400], 16, 1, D, dtype, 9, DEV)
    q = au.queries(1, 1, D, dtype, 10, DEV)
    q[:] = 0.0
    q[..., 0] = 8.0
    where = oatt.slots(c["page_indices"].tolist(), c["page_indptr"].tolist(), c["last_page_len"].tolist(), 16, 0)
    # scores 8 k / 8 = k, from -cap / 2 to cap / 2
    for (p, i), k in zip(where, np.linspace(-cap / 2, cap / 2, 400)):
        c["k_cache"][p, i, 0, 0] = float(k)
    for call, short in ((lambda: lib().attention_decode_paged(q, **c, softcap=cap, return_lse=True), False),
                        (lambda: lib().attention_prefill_paged(q, au.i32([0, 1], DEV), **c, softcap=cap, return_lse=True), cap <= 64)):
        got = call()
        torch.cuda.synchronize()
        check(got, q, None, c, D, dtype, cap, short)
