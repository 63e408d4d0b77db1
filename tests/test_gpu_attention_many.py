"""Chunk attention of batches so large that the plan keeps its sequences in memory
(over 1,024), among them empty ones, at every head size."""

import pytest
import torch

import attention_util as au
from oracle import attention as oatt

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("D,dtype,B", [(64, HF, 1025), (128, BF, 1024), (128, HF, 1500), (256, BF, 2100)])
def test_many_sequences(D, dtype, B):
    import paged_recurrent_state_amd as gdn
    new = [(i * 7) % 4 for i in range(B)]
    past = [(i * 13) % 23 for i in range(B)]
    new[B // 2], past[B - 1] = 300, 500
    c = au.batch([a + b for a, b in zip(new, past)], 8, 1, D, dtype, D, DEV)
    q = au.queries(sum(new), 2, D, dtype, D + 1, DEV)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    o, lse = gdn.attention_prefill_paged(q, au.i32(cu, DEV), **c, return_lse=True)
    torch.cuda.synchronize()
    ref = oatt.attention_paged(au.f64(q), cu, au.f64(c["k_cache"]), au.f64(c["v_cache"]), c["page_indices"].tolist(),
                               c["page_indptr"].tolist(), 8, c["last_page_len"].tolist())
    au.check_attention(o, lse, ref, D, dtype)
