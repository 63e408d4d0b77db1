"""Pins of the attention layers' oracle: closed forms, invariants of the rotation,
and torch's softmax in 64 bits (CPU only)."""

import math

import numpy as np
import pytest
import torch

from oracle import attention as oatt

EPS = 1e-12  # a few thousand roundings of 2^-53 of numbers near 1


def test_frequencies():
    assert np.allclose(oatt.frequencies(4), [1.0, 0.01], atol=EPS)
    assert np.allclose(oatt.frequencies(4, base=100.0, scaling="linear", factor=4.0), [0.25, 0.025], atol=EPS)
    plain = oatt.frequencies(64)
    f = oatt.frequencies(64, scaling="base", factor=8.0)
    assert abs(f[0] - plain[0]) < EPS and abs(f[-1] - plain[-1] / 8.0) < EPS
    # pairs that turn once or less over 4,096 tokens slow down by the factor, four times or more not at
    # all, and one in the middle (2.5 turns) by the mean of the two
    f = oatt.frequencies(64, scaling="bands", factor=8.0, original=4096.0)
    turns = 4096.0 * plain / (2 * math.pi)
    assert np.allclose(f[turns <= 1], plain[turns <= 1] / 8.0, atol=EPS)
    assert np.allclose(f[turns >= 4], plain[turns >= 4], atol=EPS)
    g = oatt.frequencies(2, scaling="bands", factor=8.0, original=5 * math.pi)
    assert abs(g[0] - (1 / 8 + 1) / 2) < EPS


def test_table():
    t = oatt.table(5, 4, magnitude=2.0)
    assert np.allclose(t[0], [2, 2, 0, 0], atol=EPS)
    assert np.allclose(t[3], 2 * np.array([math.cos(3), math.cos(0.03), math.sin(3), math.sin(0.03)]), atol=EPS)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate(interleaved):
    r = np.random.default_rng(0)
    # a quarter turn of the first pair takes (a, b) to (-b, a) and leaves the rest
    tab = np.array([[0.0, 1.0, 1.0, 0.0]])
    x = r.standard_normal((1, 2, 6))
    y = oatt.rotate(x, tab, [0], interleaved)
    a, b = (0, 1) if interleaved else (0, 2)
    want = x.copy()
    want[..., a], want[..., b] = -x[..., b], x[..., a]
    assert np.allclose(y, want, atol=EPS)
    # the transposed map takes it back, and products depend on the distance alone
    tab = oatt.table(40, 6)
    assert np.allclose(oatt.rotate(y, tab[:1], [0], interleaved, transposed=True), y, atol=EPS)
    q, k = r.standard_normal((2, 1, 1, 8))

    def product(m, n):
        return (oatt.rotate(q, tab, [m], interleaved) * oatt.rotate(k, tab, [n], interleaved)).sum()

    assert abs(product(11, 4) - product(37, 30)) < EPS
    z = oatt.rotate(oatt.rotate(q, tab, [23], interleaved), tab, [23], interleaved, transposed=True)
    assert np.allclose(z, q, atol=EPS)


def test_slots():
    assert oatt.slots([7, 3, 9], [0, 2, 2, 3], [1, 0, 4], 4, 0) == [(7, 0), (7, 1), (7, 2), (7, 3), (3, 0)]
    assert oatt.slots([7, 3, 9], [0, 2, 2, 3], [1, 0, 4], 4, 1) == []
    assert oatt.slots([7, 3, 9], [0, 2, 2, 3], [1, 0, 4], 4, 2) == [(9, 0), (9, 1), (9, 2), (9, 3)]


@pytest.mark.parametrize("window,causal,softcap", [(0, True, 0.0), (3, True, 0.0), (0, False, 5.0), (0, True, 2.0)])
def test_softmax_rows(window, causal, softcap):
    r = np.random.default_rng(1)
    n, L, D = 5, 12, 8
    q, k, v = r.standard_normal((n, D)), r.standard_normal((L, D)), r.standard_normal((L, D))
    pos = list(range(L - n, L))
    o, lse = oatt.softmax_rows(q, k, v, pos, softcap=softcap, window=window, causal=causal)[:2]
    x = torch.tensor(q @ k.T / math.sqrt(D))
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    t, j = torch.tensor(pos)[:, None], torch.arange(L)[None, :]
    hidden = (j > t) if causal else torch.zeros(n, L, dtype=torch.bool)
    if window:
        hidden = hidden | (j <= t - window)
    x = x.masked_fill(hidden, -math.inf)
    assert np.allclose(o, (torch.softmax(x, dim=1) @ torch.tensor(v)).numpy(), atol=EPS)
    assert np.allclose(lse, torch.logsumexp(x, dim=1).numpy(), atol=EPS)


def test_softmax_rows_without_keys():
    o, lse = oatt.softmax_rows(np.ones((2, 4)), np.ones((3, 4)), np.ones((3, 4)), [-1, 0])[:2]
    assert (o[0] == 0).all() and lse[0] == -math.inf
    assert np.allclose(o[1], 1.0, atol=EPS) and abs(lse[1] - 2.0) < EPS


def test_attention_paged_equals_dense():
    r = np.random.default_rng(2)
    page, H, Hk, D = 4, 4, 2, 8
    lens, new = [6, 0, 5], [2, 0, 5]
    idx, ptr, lpl = [4, 1, 0, 2], [0, 2, 2, 4], [2, 0, 1]
    kc, vc = r.standard_normal((2, 5, page, Hk, D))
    cu = [0, 2, 2, 7]
    q = r.standard_normal((7, H, D))
    res = oatt.attention_paged(q, cu, kc, vc, idx, ptr, page, lpl)
    o, lse = res[0], res[1]
    for b in range(3):
        where = oatt.slots(idx, ptr, lpl, page, b)
        for h in range(H):
            if not where:
                continue
            k = np.stack([kc[p, i, h // 2] for p, i in where])
            v = np.stack([vc[p, i, h // 2] for p, i in where])
            rows = slice(cu[b], cu[b + 1])
            a, c = oatt.softmax_rows(q[rows, h], k, v, list(range(lens[b] - new[b], lens[b])))[:2]
            assert np.allclose(o[rows, h], a, atol=EPS) and np.allclose(lse[rows, h], c, atol=EPS)
