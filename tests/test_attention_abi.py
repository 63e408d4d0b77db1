"""Refusals of the attention layers' entry points, before any launch (CPU): the
C ABI's statuses and the binding's exceptions."""

import ctypes as C

import pytest
import torch

import attention_util as au
import paged_recurrent_state_amd as gdn
from paged_recurrent_state_amd import _lib
from paged_recurrent_state_amd._lib import _AttentionC, _CacheC, _RopeC, _RowsC, _ScalingC

OK, EINVAL, EUNSUPPORTED, EWORKSPACE = 0, -1, -2, -4
FAKE = 0x1000  # an address the calls below never reach


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, page_stride=2 * 16 * 128, token_stride=2 * 128, head_stride=128, page_size=16,
             num_seqs=2, page_indices=FAKE, page_indptr=FAKE, last_page_len=FAKE)
    f.update(kw)
    return _CacheC(**f)


def dims(**kw):
    f = dict(num_q_heads=4, num_kv_heads=2, head_dim=128, dtype=0, scale=0.0, softcap=0.0, window=0, causal=1)
    f.update(kw)
    return _AttentionC(**f)


def rows(ts=4 * 128, hs=128, data=FAKE):
    return _RowsC(data, ts, hs)


def prefill(lib, d=None, c=None, q=None, out=None, cu=FAKE, T=5, ws=FAKE, nbytes=1 << 40):
    return lib.gdn_attention_prefill_paged(d or dims(), q or rows(), cu, T, c or cache(), out or rows(), None, ws,
                                           nbytes, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(num_q_heads=0), EINVAL, "head counts"),
    (dict(num_kv_heads=-1), EINVAL, "head counts"),
    (dict(num_q_heads=5), EUNSUPPORTED, "multiple"),
    (dict(head_dim=96), EUNSUPPORTED, "head_dim"),
    (dict(dtype=2), EUNSUPPORTED, "16-bit"),
    (dict(dtype=7), EINVAL, "dtype"),
    (dict(window=-1), EINVAL, "window"),
    (dict(scale=float("nan")), EINVAL, "finite"),
    (dict(softcap=float("inf")), EINVAL, "finite"),
])
def test_attention_dims(lib, kw, code, text):
    assert prefill(lib, dims(**kw)) == code
    assert text in lib.gdn_last_error().decode()
    assert lib.gdn_attention_decode_paged(dims(**kw), rows(), cache(), rows(), None, FAKE, 1 << 40, None) == code
    assert lib.gdn_attention_workspace_size(dims(**kw), 10, 2) == 0


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(page_indices=None), dict(page_indptr=None),
                                dict(last_page_len=None), dict(page_size=0), dict(num_seqs=-1),
                                dict(k=FAKE + 2), dict(v=FAKE + 8), dict(page_stride=100), dict(token_stride=100),
                                dict(head_stride=4)])
def test_attention_cache(lib, kw):
    assert prefill(lib, c=cache(**kw)) == EINVAL
    assert lib.gdn_last_error()


def test_attention_rows_and_sizes(lib):
    assert prefill(lib, q=rows(data=None)) == EINVAL
    assert prefill(lib, q=rows(data=FAKE + 2)) == EINVAL
    assert prefill(lib, q=rows(ts=3)) == EINVAL
    assert prefill(lib, out=rows(hs=3)) == EINVAL
    assert prefill(lib, cu=None) == EINVAL
    assert prefill(lib, T=-1) == EINVAL
    assert prefill(lib, T=1 << 31) == EINVAL
    assert prefill(lib, T=(1 << 30) + 5) == EINVAL  # rows of a kv-head: twice that
    assert prefill(lib, ws=None) == EWORKSPACE
    assert prefill(lib, nbytes=0) == EWORKSPACE
    null = C.POINTER(_RowsC)()
    assert lib.gdn_attention_prefill_paged(dims(), null, FAKE, 5, cache(), rows(), None, FAKE, 1 << 40, None) == EINVAL
    assert prefill(lib, T=0) == OK                       # nothing to do, nothing launched
    assert prefill(lib, c=cache(num_seqs=0)) == OK


def test_workspace_never_decreases(lib):
    for d in (dims(), dims(head_dim=64, num_q_heads=2), dims(head_dim=256, num_q_heads=32)):
        for B in (1, 3, 300):
            sizes = [lib.gdn_attention_workspace_size(d, T, B) for T in (0, 1, 5, 100, 256, 1000, 5000, 100000)]
            assert sizes == sorted(sizes) and sizes[0] >= 0
        for T in (1, 600, 100000):
            sizes = [lib.gdn_attention_workspace_size(d, T, B) for B in (1, 2, 7, 64, 65, 300, 5000)]
            assert sizes == sorted(sizes)


def rope_call(lib, r, D=128, Hq=4, Hk=2, T=3, pos=FAKE, dtype=0, idx=0, q=None, k=None):
    return lib.gdn_rope(r, dtype, D, Hq, Hk, T, pos, idx, q or rows(), k or rows(), rows(), rows(), None)


def test_rope_refusals(lib):
    good = dict(table=FAKE, table_rows=10, rot_dim=64, interleaved=0, transposed=0)
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=130), dict(table=None), dict(table_rows=-1)):
        assert rope_call(lib, _RopeC(**{**good, **kw})) == EINVAL
        assert "rope" in lib.gdn_last_error().decode()
    r = _RopeC(**good)
    assert rope_call(lib, r, D=0) == EINVAL
    assert rope_call(lib, r, Hq=-1) == EINVAL
    assert rope_call(lib, r, T=-1) == EINVAL
    assert rope_call(lib, r, pos=None) == EINVAL
    assert rope_call(lib, r, dtype=3) == EINVAL
    assert rope_call(lib, r, idx=2) == EINVAL
    assert rope_call(lib, r, q=rows(data=None)) == EINVAL
    assert rope_call(lib, r, T=0) == OK
    assert lib.gdn_rope(None, 0, 128, 4, 2, 3, FAKE, 0, rows(), rows(), rows(), rows(), None) == EINVAL


def test_append_refusals(lib):
    def call(D=128, Hk=2, cu=FAKE, T=3, c=None, k=None, rope=None, q=None, qo=None, dtype=0):
        return lib.gdn_kv_append_paged(rope, dtype, D, 4, Hk, cu, T, k or rows(), rows(), c or cache(), q, qo, None)

    assert call(D=0) == EINVAL
    assert call(Hk=0) == EINVAL
    assert call(T=-2) == EINVAL
    assert call(cu=None) == EINVAL  # 3 tokens in 2 sequences
    assert call(c=cache(page_size=0)) == EINVAL
    assert call(c=cache(k=None)) == EINVAL
    assert call(k=rows(data=None)) == EINVAL
    assert call(q=rows()) == EINVAL  # q without q_out
    assert call(dtype=9) == EINVAL
    assert call(rope=_RopeC(FAKE, 10, 7, 0, 0)) == EINVAL
    assert call(T=0) == OK


def test_table_refusals(lib):
    good = dict(scaling=0, base=10000.0, factor=1.0, original=0.0, low_turns=1.0, high_turns=4.0, magnitude=1.0)
    for kw in (dict(scaling=4), dict(scaling=-1), dict(base=0.0), dict(base=-1.0), dict(scaling=1, factor=0.0),
               dict(magnitude=float("inf")), dict(scaling=3, factor=2.0), dict(scaling=3, original=64.0, high_turns=1.0),
               dict(base=float("nan"))):
        assert lib.gdn_rope_table(_ScalingC(**{**good, **kw}), FAKE, 10, 64, None) == EINVAL, kw
    g = _ScalingC(**good)
    assert lib.gdn_rope_table(g, FAKE, 10, 63, None) == EINVAL
    assert lib.gdn_rope_table(g, FAKE, -1, 64, None) == EINVAL
    assert lib.gdn_rope_table(g, None, 10, 64, None) == EINVAL
    assert lib.gdn_rope_table(_ScalingC(**{**good, "scaling": 2, "factor": 2.0}), FAKE, 10, 2, None) == EINVAL
    assert lib.gdn_rope_table(g, None, 0, 64, None) == OK


def test_binding_refuses_host_tensors():
    bf = torch.bfloat16
    c = au.batch([5, 9], 16, 2, 64, bf, 0)
    q, k = au.queries(2, 4, 64, bf, 1), au.queries(2, 2, 64, bf, 2)
    tab = torch.zeros(16, 64)
    for call in (lambda: gdn.rope_table(4, 64, device="cpu"),
                 lambda: gdn.rope(q, k, tab, torch.arange(2)),
                 lambda: gdn.rope_backward(q, k, tab, torch.arange(2)),
                 lambda: gdn.kv_append_paged(k, k, None, **c),
                 lambda: gdn.attention_prefill_paged(q, au.i32([0, 1, 2]), **c),
                 lambda: gdn.attention_decode_paged(q, **c)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_binding_refusals_on_the_gpu():
    bf, dev = torch.bfloat16, "cuda"
    c = au.batch([5, 9], 16, 2, 64, bf, 0, dev)
    q, k = au.queries(2, 4, 64, bf, 1, dev), au.queries(2, 2, 64, bf, 2, dev)
    tab = torch.zeros(16, 64, device=dev)
    cu = au.i32([0, 1, 2], dev)
    bad = [
        (TypeError, lambda: gdn.attention_decode_paged(q.half(), **c)),
        (gdn.GDNError, lambda: gdn.attention_decode_paged(q.float(), **{**c, "k_cache": c["k_cache"].float(),
                                                                       "v_cache": c["v_cache"].float()})),
        (ValueError, lambda: gdn.attention_decode_paged(q[:1], **c)),
        (ValueError, lambda: gdn.attention_decode_paged(q, **{**c, "page_size": 8})),
        (ValueError, lambda: gdn.attention_decode_paged(q, **{**c, "v_cache": c["v_cache"][:1]})),
        (ValueError, lambda: gdn.attention_decode_paged(q, **{**c, "v_cache": c["v_cache"].transpose(1, 2).contiguous().transpose(1, 2)})),
        (ValueError, lambda: gdn.attention_prefill_paged(q, cu[:2], **c)),
        (TypeError, lambda: gdn.attention_prefill_paged(q, cu.long(), **c)),
        (gdn.GDNError, lambda: gdn.attention_decode_paged(q[:, :3], **c)),
        (gdn.GDNError, lambda: gdn.attention_decode_paged(q, **c, window=-1)),
        (ValueError, lambda: gdn.attention_decode_paged(q, **c, out=torch.empty(2, 4, 32, dtype=bf, device=dev))),
        (ValueError, lambda: gdn.kv_append_paged(k[:, :1], k[:, :1], None, **c)),
        (TypeError, lambda: gdn.kv_append_paged(k, k.half(), None, **c)),
        (gdn.GDNError, lambda: gdn.kv_append_paged(k[:1], k[:1], None, **c)),
        (TypeError, lambda: gdn.rope(q, None, tab.double(), torch.arange(2, device=dev))),
        (TypeError, lambda: gdn.rope(q, None, tab, torch.arange(2, device=dev).float())),
        (ValueError, lambda: gdn.rope(q, None, tab, torch.arange(3, device=dev))),
        (ValueError, lambda: gdn.rope(q, k[:1], tab, torch.arange(2, device=dev))),
        (ValueError, lambda: gdn.rope(q.transpose(1, 2), None, tab, torch.arange(2, device=dev))),
        (gdn.GDNError, lambda: gdn.rope(q, None, torch.zeros(4, 66, device=dev), torch.arange(2, device=dev))),
        (ValueError, lambda: gdn.rope_table(4, 64, scaling="other")),
        (gdn.GDNError, lambda: gdn.rope_table(4, 63)),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"call {i} was not refused")
