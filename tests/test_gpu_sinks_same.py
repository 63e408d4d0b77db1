"""A window and sinks that together leave nothing out give what no window gives: each value within its bound of the
64-bit one, so the two within twice that, whatever the sign."""

import numpy as np
import pytest
import torch

import attention_util as au
from oracle import attention as oatt

pytestmark = pytest.mark.gpu
DEV, BF, HF = "cuda", torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(100, 200), (1, 260), (130, 130), (260, 1)])
def test_nothing_left_out(dtype, D, window, sinks):
    import paged_recurrent_state_amd as m
    new, past = [60, 3], [200, 10]
    c = au.batch([a + b for a, b in zip(new, past)], 16, 2, D, dtype, 60, DEV)
    q, cu = au.queries(63, 4, D, dtype, 61, DEV), au.i32([0, 60, 63], DEV)
    where = [c[n].tolist() if isinstance(c[n], torch.Tensor) else c[n] for n in ("page_indices", "page_indptr", "page_size",
                                                                               "last_page_len")]
    kv = [au.f64(c[n]) for n in ("k_cache", "v_cache")]
    for rows, cus, call in ((q, cu.tolist(), lambda **kw: m.attention_prefill_paged(q, cu, **c, return_lse=True, **kw)),
                            (q[[59, 62]], [0, 1, 2], lambda **kw: m.attention_decode_paged(q[[59, 62]].contiguous(), **c, return_lse=True, **kw))):
        ref = oatt.attention_paged(au.f64(rows), cus, *kv, *where)
        a, b = call(), call(window=window, sinks=sinks)
        eo, el = au.attention_bounds(ref, D, dtype)
        au.check_attention(*a, ref, D, dtype)
        au.check_attention(*b, ref, D, dtype)
        assert (np.abs(au.f64(a[0]) - au.f64(b[0])) <= 2 * eo).all() and (np.abs(au.f64(a[1]) - au.f64(b[1])) <= 2 * el).all()
