"""Refusals of the norms', the 8-bit cache's and the sinks' entry points, before any
launch (CPU): the C ABI's statuses and the binding's exceptions."""

import pytest
import torch

import attention_util as au
import paged_recurrent_state_amd as gdn
from paged_recurrent_state_amd import _lib
from paged_recurrent_state_amd._lib import _AttentionC, _CacheC, _NormC, _RopeC, _RowsC, _ScalesC

OK, EINVAL, EUNSUPPORTED, EWORKSPACE = 0, -1, -2, -4
FAKE = 0x10000  # an address the calls below never reach
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def rows(ts=4 * 128, hs=128, data=FAKE):
    return _RowsC(data, ts, hs)


def norm(**kw):
    f = dict(q_weight=FAKE, k_weight=FAKE, weight_dtype=0, eps=1e-6, offset=0.0)
    f.update(kw)
    return _NormC(**f)


def rope(**kw):
    f = dict(table=FAKE, table_rows=10, rot_dim=64, interleaved=0, transposed=0)
    f.update(kw)
    return _RopeC(**f)


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, page_stride=2 * 64 * 128, token_stride=2 * 128, head_stride=128, page_size=64, num_seqs=2,
             page_indices=FAKE, page_indptr=FAKE, last_page_len=FAKE)
    f.update(kw)
    return _CacheC(**f)


def scales(**kw):
    f = dict(k=FAKE, v=FAKE, page_stride=8, block_stride=2, head_stride=1, block=16)
    f.update(kw)
    return _ScalesC(**f)


def norm_rope(lib, n, r=None, D=128, Hq=4, Hk=2, T=3, dtype=0):
    return lib.gdn_norm_rope(n, r or rope(), dtype, D, Hq, Hk, T, FAKE, 0, rows(), rows(), rows(), rows(), None)


def backward(lib, n, r=None, D=128, Hq=4, Hk=2, T=3, dtype=0, gw=FAKE, ws=FAKE, size=1 << 40, dx=FAKE << 8, ts=4 * 128):
    return lib.gdn_norm_rope_backward(n, r or rope(), dtype, D, Hq, Hk, T, FAKE, 0, rows(), rows(), rows(data=FAKE << 4),
                                      rows(data=FAKE << 4), rows(ts, data=dx), rows(ts, data=FAKE << 12), gw, FAKE, ws, size, None)


def append(lib, n=None, r=None, sc=None, c=None, dtype=0, D=128, k=None, T=2):
    return lib.gdn_kv_append_paged_ext(n, r, dtype, D, 4, 2, None, T, k or rows(2 * 128), rows(2 * 128), c or cache(), sc, None,
                                       None, None)


def read(lib, sc=None, c=None, dtype=0, D=128, k=None, T=2):
    return lib.gdn_kv_read_paged(dtype, D, 2, None, T, c or cache(), sc, k or rows(2 * 128), rows(2 * 128), None)


BAD_NORMS = [dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF), dict(offset=NAN), dict(offset=INF), dict(weight_dtype=1),
             dict(weight_dtype=7)]


@pytest.mark.parametrize("kw", BAD_NORMS)
def test_norms(lib, kw):
    for rc in (norm_rope(lib, norm(**kw)), backward(lib, norm(**kw)), append(lib, norm(**kw))):
        assert rc == EINVAL and "norm" in lib.gdn_last_error().decode()


def test_norm_weights_and_sizes(lib):
    for kw in (dict(q_weight=None), dict(k_weight=None)):
        assert norm_rope(lib, norm(**kw)) == EINVAL and backward(lib, norm(**kw)) == EINVAL
        assert "weights" in lib.gdn_last_error().decode()
    assert norm_rope(lib, None) == EINVAL and backward(lib, None) == EINVAL
    assert norm_rope(lib, norm(), D=516) == EUNSUPPORTED and backward(lib, norm(), D=516) == EUNSUPPORTED
    assert append(lib, norm(), D=516) == EUNSUPPORTED
    assert norm_rope(lib, norm(), rope(rot_dim=130)) == EINVAL
    assert norm_rope(lib, norm(), T=-1) == EINVAL and backward(lib, norm(), T=1 << 31) == EINVAL
    assert norm_rope(lib, norm(weight_dtype=2), T=0) == OK  # nothing to do, nothing launched
    assert norm_rope(lib, norm(), dtype=5) == EINVAL


def test_backward_workspace_and_rows(lib):
    need = lib.gdn_norm_rope_backward_workspace_size(128, 4, 2, 3)
    assert need >= 256 and need % 4 == 0
    assert backward(lib, norm(), ws=None) == EWORKSPACE and backward(lib, norm(), ws=FAKE + 16) == EWORKSPACE
    assert backward(lib, norm(), size=need - 1) == EWORKSPACE
    assert backward(lib, norm(), gw=None) == EINVAL
    # a gradient that lies a row behind the rows it is of
    assert backward(lib, norm(), dx=FAKE + 256) == EINVAL and "lie over" in lib.gdn_last_error().decode()
    assert backward(lib, norm(), dx=FAKE, ts=8 * 128) == EINVAL
    assert lib.gdn_norm_rope_backward_workspace_size(1024, 4, 2, 3) == 0
    assert lib.gdn_norm_rope_backward_workspace_size(128, -1, 2, 3) == 0
    sizes = [lib.gdn_norm_rope_backward_workspace_size(128, 32, 8, T) for T in (0, 1, 2, 7, 64, 1000, 100000, 1 << 30)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=FAKE + 2), dict(block=0), dict(block=8), dict(block=24),
                                dict(block=-16), dict(block=48), dict(block=128)])
def test_scales(lib, kw):
    for f in (append, read):
        assert f(lib, sc=scales(**kw)) == EINVAL and lib.gdn_last_error()


@pytest.mark.parametrize("kw", [dict(k=FAKE + 8), dict(v=FAKE + 4), dict(page_stride=100), dict(token_stride=72),
                                dict(head_stride=8), dict(page_size=0), dict(page_size=40), dict(k=None)])
def test_code_caches(lib, kw):
    for f in (append, read):
        assert f(lib, sc=scales(), c=cache(**kw)) == EINVAL and lib.gdn_last_error()


def test_appended_rows(lib):
    assert append(lib, sc=scales(), dtype=2) == EUNSUPPORTED
    assert append(lib, sc=scales(), D=96) == EUNSUPPORTED and read(lib, sc=scales(), D=32) == EUNSUPPORTED
    assert append(lib, sc=scales(), r=rope(rot_dim=66)) == EUNSUPPORTED
    assert append(lib, sc=scales(), k=rows(2 * 128, data=FAKE + 2)) == EUNSUPPORTED
    assert append(lib, sc=scales(), k=rows(257)) == EUNSUPPORTED
    assert append(lib, sc=scales(), T=5) == EINVAL  # two sequences, one token each
    assert read(lib, sc=None) == EINVAL
    assert read(lib, sc=scales(), k=rows(2 * 128, data=FAKE + 8)) == EINVAL
    assert read(lib, sc=scales(), T=3) == EINVAL and read(lib, sc=scales(), dtype=9) == EINVAL
    empty = cache(num_seqs=0)
    assert append(lib, sc=scales(), c=empty, T=0) == OK and read(lib, sc=scales(), c=empty, T=0) == OK


def test_attention(lib):
    d = _AttentionC(num_q_heads=4, num_kv_heads=2, head_dim=128, dtype=0, scale=0.0, softcap=0.0, window=8, causal=1)

    def calls(sinks=0, sc=None, c=None):
        a = lib.gdn_attention_prefill_paged_ext(d, sinks, rows(), FAKE, 5, c or cache(), sc, rows(data=FAKE << 4), None, FAKE,
                                                1 << 40, None)
        b = lib.gdn_attention_decode_paged_ext(d, sinks, rows(), c or cache(), sc, rows(data=FAKE << 4), None, FAKE, 1 << 40, None)
        return a, b

    assert calls(sinks=-1) == (EINVAL, EINVAL) and calls(sinks=(1 << 30) + 1) == (EINVAL, EINVAL)
    assert "sinks" in lib.gdn_last_error().decode()
    for kw in (dict(k=None), dict(block=24), dict(block=48), dict(v=FAKE + 1)):
        assert calls(sc=scales(**kw)) == (EINVAL, EINVAL)
    for kw in (dict(head_stride=8), dict(k=FAKE + 8)):
        assert calls(sc=scales(), c=cache(**kw)) == (EINVAL, EINVAL)
    for ts in (-256, 1 << 24):
        a = lib.gdn_attention_prefill_paged_ext(d, 0, rows(), FAKE, 5, cache(token_stride=ts), scales(), rows(data=FAKE << 4), None,
                                                FAKE, 1 << 40, None)
        assert a == EUNSUPPORTED and "token strides" in lib.gdn_last_error().decode()


# ------------------------------------------------------------------- binding

BF = torch.bfloat16
E4M3 = torch.float8_e4m3fn


def test_binding_has_no_cpu_path():
    q, w = torch.zeros(3, 2, 64, dtype=BF), torch.zeros(64, dtype=BF)
    tab, pos = torch.zeros(8, 64), torch.zeros(3, dtype=torch.int64)
    c = au.batch([5], 16, 2, 64, BF, 1)
    codes = {n: torch.zeros(c[n].shape, dtype=E4M3) for n in ("k_cache", "v_cache")}
    sc = dict(k_scale=torch.ones(3, 1, 2), v_scale=torch.ones(3, 1, 2))
    for call in (lambda: gdn.norm_rope(q, None, w, None, tab, pos),
                 lambda: gdn.norm_rope_backward(q, None, q, None, w, None, tab, pos),
                 lambda: gdn.kv_append_paged(q, q, au.i32([0, 3]), **{**c, **codes}, **sc),
                 lambda: gdn.kv_read_paged(au.i32([0, 3]), 3, **{**c, **codes}, **sc),
                 lambda: gdn.attention_decode_paged(q[:1], **{**c, **codes}, **sc),
                 lambda: gdn.attention_prefill_paged(q, au.i32([0, 3]), **c, window=2, sinks=1)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()


def test_helpers_of_the_binding():
    """The argument checks behind the calls, on CPU tensors."""
    from paged_recurrent_state_amd import _attention as a
    cpu = torch.device("cpu")
    kc = torch.zeros(4, 64, 2, 64, dtype=E4M3)
    sc = torch.ones(4, 4, 2)
    got = a._scales(sc, sc.clone(), kc, 64, cpu)
    assert (got.block, got.page_stride, got.block_stride, got.head_stride) == (16, 8, 2, 1)
    heads_first = torch.ones(4, 2, 2).transpose(1, 2)
    assert a._scales(heads_first, heads_first.clone(), kc, 64, cpu).block == 32
    for k, v, err in ((None, sc, ValueError), (sc, None, ValueError), (sc.double(), sc, TypeError), (sc, sc.half(), TypeError),
                      (sc[:3], sc, ValueError), (sc, sc[:, :2], ValueError), (torch.ones(4, 5, 2), torch.ones(4, 5, 2), ValueError),
                      (torch.ones(4, 0, 2), torch.ones(4, 0, 2), ValueError), (sc[..., None], sc, ValueError), ([1.0], sc, TypeError),
                      (sc, torch.ones(4, 2, 4).transpose(1, 2), ValueError)):
        with pytest.raises(err):
            a._scales(k, v, kc, 64, cpu)
    w = torch.ones(64, dtype=BF)
    assert a._norm(w, None, 1e-6, 0.0, BF, 64, cpu).weight_dtype == 0
    assert a._norm(None, w.float(), 1e-6, 0.0, BF, 64, cpu).weight_dtype == 2
    for q, k, err in ((w[:32], None, ValueError), (w, w.float(), TypeError), (w.half(), None, TypeError), ([1.0], None, TypeError),
                      (torch.ones(128, dtype=BF)[::2], None, ValueError), (w[None], None, ValueError)):
        with pytest.raises(err):
            a._norm(q, k, 1e-6, 0.0, BF, 64, cpu)
