"""The norm's gradient writes the queries' rows while it reads and writes the keys': rows of one that share memory
with the other's are refused, parts of one buffer are not (CPU: calls that get as far as the workspace, which is
missing, were not refused)."""

import itertools

import numpy as np
import pytest

from paged_recurrent_state_amd import _lib
from paged_recurrent_state_amd._lib import _NormC, _RopeC, _RowsC

EINVAL, EWORKSPACE = -1, -4
FAKE = 1 << 30  # an address the calls below never reach
SIZE = 2        # of a value
D = 64


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def call(lib, T, Hq, Hk, rows):
    """rows: six (offset in values, token stride, head stride), of q, k, their outputs' gradients and their gradients."""
    r = [_RowsC(FAKE + SIZE * at, ts, hs) for at, ts, hs in rows]
    norm, rope = _NormC(FAKE, FAKE, 0, 1e-6, 0.0), _RopeC(FAKE, 10, 32, 0, 0)
    return lib.gdn_norm_rope_backward(norm, rope, 0, D, Hq, Hk, T, FAKE, 0, *r, FAKE, FAKE, None, 0, None)


def values_of(rows, T, H):
    at, ts, hs = rows
    first = at + ts * np.arange(T)[:, None] + hs * np.arange(H)[None]
    return set((first[..., None] + np.arange(D)).ravel().tolist())


APART = [(i << 20, 4 * D, D) for i in range(6)]


@pytest.mark.parametrize("grad,other", [(4, 1), (4, 3), (4, 5), (5, 0), (5, 2), (5, 4)])
@pytest.mark.parametrize("shift", [0, D - 1, 3 * D, 8 * D + 5])
def test_gradients_over_the_other_heads_rows(lib, grad, other, shift):
    assert call(lib, 3, 4, 4, APART) == EWORKSPACE
    for sign in (1, -1):
        rows = list(APART)
        rows[grad] = (rows[other][0] + sign * shift, 4 * D, D)
        assert call(lib, 3, 4, 4, rows) == EINVAL and "must not share memory" in lib.gdn_last_error().decode()


@pytest.mark.parametrize("Hq,Hk", [(4, 2), (4, 1), (1, 1), (2, 4)])
@pytest.mark.parametrize("heads_first", [False, True])
def test_parts_of_one_buffer(lib, Hq, Hk, heads_first):
    """q, k (and v) as they come out of one projection, their gradients over them or in a buffer of the same form."""
    T, H = 5, Hq + 2 * Hk
    ts, hs = (D, T * D) if heads_first else (H * D, D)
    qk = [(0, ts, hs), (Hq * hs, ts, hs)]
    out = [(x + (1 << 20), a, b) for x, a, b in qk]
    other = [(x + (1 << 21), a, b) for x, a, b in qk]
    for grads in (qk, out, other):
        assert call(lib, T, Hq, Hk, [*qk, *out, *grads]) == EWORKSPACE
    # (a single head's stride is nothing)
    if Hk == 1:
        assert call(lib, T, Hq, Hk, [qk[0], (qk[1][0], ts, 7), out[0], (out[1][0], ts, 0), other[0], (other[1][0], ts, -9)]) == EWORKSPACE
    # the keys' a head earlier: the last of the queries'
    assert call(lib, T, Hq, Hk, [*qk, *out, other[0], (other[1][0] - hs, ts, hs)]) == EINVAL


def test_against_every_value(lib):
    """Equal strides: refused if a value of one is a value of the other, and not otherwise."""
    rng, seen = np.random.default_rng(0), set()
    for _ in range(600):
        T, Hq, Hk = (int(x) for x in rng.integers(1, 8, 3))
        ts, hs = (int(x) for x in rng.permutation([int(rng.integers(1, 28)) * 16, int(rng.integers(1, 4)) * D]))
        a = (1 << 21, ts, hs)
        b = ((1 << 21) + int(rng.integers(-30, 31)) * 32, ts, hs)
        rows = [APART[0], APART[1], (5 << 21, 4 * D, D), (6 << 21, 4 * D, D), a, b]
        shared = bool(values_of(a, T, Hq) & values_of(b, T, Hk))
        assert (call(lib, T, Hq, Hk, rows) == EINVAL) == shared, (T, Hq, Hk, a, b)
        seen.add(shared)
    assert seen == {False, True}


def test_no_rows_share_nothing(lib):
    rows = [(0, 4 * D, D)] * 6
    for T, Hq, Hk in itertools.product((0, 3), (0, 4), (0, 4)):
        want = 0 if not Hq + Hk else EINVAL if T and Hq and Hk else EWORKSPACE
        assert call(lib, T, Hq, Hk, rows) == want
