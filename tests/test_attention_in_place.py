"""Output rows over the query rows: a chunk's call refuses them, whatever part they
share, and takes interleaved parts of one buffer; single tokens may be in place."""

import itertools

import pytest
import torch

import attention_util as au
import paged_recurrent_state_amd as gdn
from paged_recurrent_state_amd import _lib
from paged_recurrent_state_amd._lib import _AttentionC, _CacheC, _RowsC

EINVAL = -1
FAKE = 1 << 20  # addresses the calls below never reach


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def refusal(lib, q, out, T, H=4, D=64, decode=False):
    """The message of a call that is refused by the last check of its arguments."""
    d = _AttentionC(H, 2, D, 0, 0.0, 0.0, 0, 1)
    c = _CacheC(FAKE, FAKE, 2 * 16 * D, 2 * D, D, 16, T if decode else 2, FAKE, FAKE, FAKE)
    if decode:
        rc = lib.gdn_attention_decode_paged(d, _RowsC(*q), c, _RowsC(*out), None, FAKE, 1 << 40, None)
    else:
        rc = lib.gdn_attention_prefill_paged(d, _RowsC(*q), FAKE, T, c, _RowsC(*out), None, FAKE, 1 << 40, None)
    assert rc == EINVAL
    return lib.gdn_last_error().decode()


Q = (FAKE, 4 * 64, 64)  # dense rows of 4 heads of 64


@pytest.mark.parametrize("out,T", [
    (Q, 5), (Q, 1),
    ((FAKE + 2 * 64 * 4, 4 * 64, 64), 5),             # a token later
    ((FAKE + 2 * 64, 4 * 64, 64), 1),                 # a head later
    ((FAKE + 16, 4 * 64, 64), 5),                     # within a row
    ((FAKE - 2 * 64 * 4 * 4 - 2 * 64, 4 * 64, 64), 5),  # its last rows
    ((FAKE, 64, 5 * 64), 5),                          # the same block, heads first
    ((FAKE + 2 * 64 * 4 * 4, -4 * 64, 64), 5),        # backwards
    ((FAKE, 0, 64), 5),
])
def test_chunks_refuse_outputs_over_the_queries(lib, out, T):
    assert "share memory" in refusal(lib, Q, out, T)
    assert "share memory" in refusal(lib, out, Q, T)


def test_single_tokens_refuse_all_but_the_queries_themselves(lib):
    assert "share memory" in refusal(lib, Q, (FAKE + 2 * 64, 4 * 64, 64), 5, decode=True)
    assert "share memory" in refusal(lib, Q, (FAKE, 64, 5 * 64), 5, decode=True)


def overlap(q, out, T, H, D):
    """By every byte."""
    rows = [{(r[0] + 2 * (t * r[1] + h * r[2])) // 2 + d for t, h, d in itertools.product(range(T), range(H), range(D))}
            for r in (q, out)]
    return bool(rows[0] & rows[1])


@pytest.mark.gpu
def test_interleaved_parts_of_one_buffer():
    """Parts of a projection's output that lie between each other: with equal strides no call is refused that
    shares nothing."""
    dev, bf, D, H, T = "cuda", torch.bfloat16, 64, 4, 6
    c = au.batch([9, 30], 16, 2, D, bf, 0, dev)
    cu = au.i32([0, 2, T], dev)
    buf = au.queries(2 * T, 3 * H, D, bf, 1, dev)
    keep = buf.clone()
    ref = gdn.attention_prefill_paged(keep[:T, :H].contiguous(), cu, **c)
    views = [buf[:T, H:2 * H], buf[T:, :H], buf[::2, :H], buf.view(T, 2, 3 * H, D)[:, 1, H:2 * H], buf[:T, ::3], buf[1:T + 1, :H]]
    base = buf[:T, :H]
    where = lambda t: (t.data_ptr(), t.stride(0), t.stride(1))
    for v in views:
        if overlap(where(base), where(v), T, H, D):
            with pytest.raises(gdn.GDNError, match="share memory"):
                gdn.attention_prefill_paged(base, cu, **c, out=v)
        elif v.stride() == base.stride():
            buf.copy_(keep)
            gdn.attention_prefill_paged(base, cu, **c, out=v)
            torch.cuda.synchronize()
            assert torch.equal(v, ref)
    assert [overlap(where(base), where(v), T, H, D) for v in views] == [False, False, True, False, True, True]


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16), (256, torch.bfloat16)])
def test_single_tokens_in_place(D, dtype):
    lens = [1, 0, 700, 33, 5000]
    c = au.batch(lens, 16, 2, D, dtype, 2, "cuda")
    for G in (1, 4, 20):
        q = au.queries(len(lens), 2 * G, D, dtype, 3, "cuda", 2.0)
        ref, lse = gdn.attention_decode_paged(q, **c, return_lse=True)
        got, lse2 = gdn.attention_decode_paged(q, **c, out=q, return_lse=True)
        torch.cuda.synchronize()
        assert got.data_ptr() == q.data_ptr() and torch.equal(got, ref) and torch.equal(lse, lse2)
