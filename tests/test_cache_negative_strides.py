"""Caches whose pages or tokens lie backwards in memory are refused by every call that takes one (CPU): the kernels
tell tokens that are not there by a negative offset, and passed over such pages without a word."""

import pytest

from paged_recurrent_state_amd import _lib
from paged_recurrent_state_amd._lib import _AttentionC, _CacheC, _RowsC, _ScalesC

EUNSUPPORTED, EWORKSPACE = -2, -4
FAKE = 1 << 24  # an address the calls below never reach


def calls(lib, c, coded):
    """Statuses of the calls over cache c; those that reach the workspace, which is missing, took it."""
    rows, out = _RowsC(FAKE, 2 * 64, 64), _RowsC(2 * FAKE, 2 * 64, 64)
    sc = _ScalesC(FAKE, FAKE, 8, 2, 1, 16) if coded else None
    d = _AttentionC(2, 2, 64, 0, 0.0, 0.0, 8, 1)
    yield lib.gdn_attention_decode_paged_ext(d, 1, rows, c, sc, out, None, None, 0, None)
    yield lib.gdn_attention_prefill_paged_ext(d, 1, rows, FAKE, 3, c, sc, out, None, None, 0, None)


def appends(lib, c, coded):
    rows = _RowsC(FAKE, 2 * 64, 64)
    sc = _ScalesC(FAKE, FAKE, 8, 2, 1, 16) if coded else None
    yield lib.gdn_kv_append_paged_ext(None, None, 0, 64, 0, 2, None, 2, rows, rows, c, sc, None, None, None)
    if coded:
        yield lib.gdn_kv_read_paged(0, 64, 2, None, 2, c, sc, rows, rows, None)
    else:
        yield lib.gdn_kv_append_paged(None, 0, 64, 0, 2, None, 2, rows, rows, c, None, None, None)


def cache(page=32, **kw):
    f = dict(k=FAKE, v=FAKE, page_stride=2 * 64 * 64, token_stride=2 * 64, head_stride=64, page_size=page, num_seqs=2,
             page_indices=FAKE, page_indptr=FAKE, last_page_len=FAKE)
    f.update(kw)
    return _CacheC(**f)


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("kw", [dict(page_stride=-2 * 64 * 64), dict(token_stride=-2 * 64), dict(page_stride=-64, token_stride=-64)])
def test_refused(coded, kw):
    lib = _lib.load()
    for rc in (*calls(lib, cache(**kw), coded), *appends(lib, cache(**kw), coded)):
        assert rc == EUNSUPPORTED and "strides of 0 and more" in lib.gdn_last_error().decode()


@pytest.mark.parametrize("kw", [dict(), dict(head_stride=-64), dict(page_stride=0), dict(token_stride=0)])
def test_taken(kw):
    lib = _lib.load()
    for coded in (False, True):
        assert set(calls(lib, cache(**kw), coded)) == {EWORKSPACE}
    # (pages of one token have no step between tokens)
    assert set(calls(lib, cache(1, token_stride=-2 * 64), False)) == {EWORKSPACE}
