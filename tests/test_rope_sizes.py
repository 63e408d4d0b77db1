"""Heads and head sizes at the limits of the rotary kernel's thread numbers (CPU:
refusals before any launch)."""

import pytest

from paged_recurrent_state_amd import _lib
from paged_recurrent_state_amd._lib import _CacheC, _RopeC, _RowsC

OK, EINVAL = 0, -1
FAKE = 1 << 20  # an address the calls below never reach


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def rows(heads, dim, off=2):
    """Rows at an address (2 bytes off) that leaves one pair a thread: head_dim - rot_dim / 2 threads a row."""
    return _RowsC(FAKE + off, heads * dim, dim)


# threads of a token: 2^32, 2^31 + 2^15, 65535 * 32769 and more
SIZES = [(65536, 65536, 2), (65536, 32770, 2), (32769, 65536, 2), (65536, 65536, 65536), (65535, 32772, 4)]


@pytest.mark.parametrize("heads,dim,rot", SIZES)
def test_rope(lib, heads, dim, rot):
    rope = _RopeC(FAKE, 10, rot, 0, 0)
    r = rows(heads, dim)
    rc = lib.gdn_rope(rope, 0, dim, heads, 0, 1, FAKE, 0, r, None, r, None, None)
    assert rc == EINVAL and "threads" in lib.gdn_last_error().decode()


@pytest.mark.parametrize("heads,dim,rot", SIZES)
def test_append(lib, heads, dim, rot):
    rope = _RopeC(FAKE, 10, rot, 0, 0)
    hk = heads // 2 - 1
    hq = heads - 2 * hk
    c = _CacheC(FAKE, FAKE, 16 * hk * dim, hk * dim, dim, 16, 1, FAKE, FAKE, FAKE)
    r, q = rows(hk, dim), rows(hq, dim)
    rc = lib.gdn_kv_append_paged(rope, 0, dim, hq, hk, None, 1, r, r, c, q, q, None)
    assert rc == EINVAL and "threads" in lib.gdn_last_error().decode()


def test_no_tokens_launch_nothing(lib):
    rope = _RopeC(FAKE, 10, 64, 0, 0)
    r = rows(64, 128)
    assert lib.gdn_rope(rope, 0, 128, 64, 0, 0, FAKE, 0, r, None, r, None, None) == OK
