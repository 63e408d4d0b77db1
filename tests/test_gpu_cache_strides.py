"""Caches one of whose dimensions has a single entry: its stride says nothing, and
neither differing nor odd ones are refused."""

import pytest
import torch

import attention_util as au
import paged_recurrent_state_amd as gdn

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def restrided(t, dim, stride):
    """The same values at the same places, with another stride of the dimension of one entry."""
    assert t.shape[dim] == 1
    s = list(t.stride())
    s[dim] = stride
    # (storage enough for what the strides claim is not needed: the dimension has one entry)
    return t.as_strided(t.shape, s, t.storage_offset())


@pytest.mark.parametrize("lens,page,Hk,dim", [([40, 9], 16, 1, 2), ([3, 5], 1, 2, 1), ([13], 16, 2, 0)])
def test_a_dimension_of_one(lens, page, Hk, dim):
    c = au.batch(lens, page, Hk, 64, BF, 0, DEV, spare=0)
    assert c["k_cache"].shape[dim] == 1
    q, k = au.queries(len(lens), 2 * Hk, 64, BF, 1, DEV), au.queries(len(lens), Hk, 64, BF, 2, DEV)
    cu = au.i32(list(range(len(lens) + 1)), DEV)

    def calls(c):
        gdn.kv_append_paged(k, k, None, **c)
        return gdn.attention_decode_paged(q, **c), gdn.attention_prefill_paged(q, cu, **c)

    want = calls(c)
    for ks, vs in ((8, 8), (64, 192), (3, 5), (0, 64)):
        other = {**c, "k_cache": restrided(c["k_cache"], dim, ks), "v_cache": restrided(c["v_cache"], dim, vs)}
        assert all(torch.equal(a, b) for a, b in zip(calls(other), want))


def test_layouts_that_differ_are_refused():
    c = au.batch([40, 9], 16, 2, 64, BF, 0, DEV)
    q = au.queries(2, 4, 64, BF, 1, DEV)
    c["v_cache"] = c["v_cache"].transpose(1, 2).contiguous().transpose(1, 2)
    with pytest.raises(ValueError, match="strides"):
        gdn.attention_decode_paged(q, **c)
