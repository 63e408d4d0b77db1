"""Pins of the oracle of the norms, of the cache of 8 bits and of sinks: torch's float8
rounding, differences and torch's gradients in 64 bits, a masked softmax."""

import math

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import norms, quantised


def test_e4m3_is_torchs_rounding():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    finite = codes[np.isfinite(codes)]
    assert np.array_equal(quantised.e4m3(finite), finite) and finite.max() == quantised.MOST
    r = np.random.default_rng(1)
    x = np.concatenate([r.standard_normal(5000) * s for s in (1e-3, 1e-2, 1.0, 100.0)])
    between = np.sort(finite)
    x = np.concatenate([x, (between[1:] + between[:-1]) / 2, [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(quantised.e4m3(x), want)
    assert np.isnan(quantised.e4m3([np.nan, np.inf])).all()


@pytest.mark.parametrize("top,scale", [(448.0, 1.0), (448.0000001, 2.0), (224.0, 0.5), (224.1, 1.0), (1.0, 2.0 ** -8),
                                       (0.875, 2.0 ** -9), (0.0, 2.0 ** -100), (1e-40, 2.0 ** -100), (3e38, 2.0 ** 120)])
def test_scale(top, scale):
    assert quantised.scale_of(top) == scale


def test_append_block_by_block():
    """Two tokens join one that is there: the scale grows, the first token's codes are rounded to it."""
    cache, scale = np.zeros((1, 16, 1, 64)), np.full((1, 1, 1), np.nan)
    rows = np.zeros((3, 1, 64))
    rows[0, 0, 0], rows[1, 0, 0], rows[2, 0, 0] = 1.1, 300.0, 2.0
    quantised.append(cache, scale, rows[:1], [1], [1], [0], [0, 1], 16, 16)
    assert scale[0, 0, 0] == 2.0 ** -8 and cache[0, 0, 0, 0] == 288  # 281.6 among steps of 32
    quantised.append(cache, scale, rows[1:], [2], [3], [0], [0, 1], 16, 16)
    assert scale[0, 0, 0] == 1.0 and cache[0, :3, 0, 0].tolist() == [1.125, 288, 2.0] and not cache[0, 3:].any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norm_gradient_is_torchs_and_differences(interleaved, offset):
    T, H, D, rot, eps = 3, 2, 8, 4, 1e-3
    r = np.random.default_rng(2)
    x, w, g = r.standard_normal((T, H, D)), r.standard_normal(D), r.standard_normal((T, H, D))
    tab, pos = oatt.table(10, rot), [0, 7, 3]
    dx, dw = norms.norm_rope_grad(g, x, w, tab, pos, eps, offset, interleaved)
    # the loss <g, R n(x)> = <R^T g, n(x)>
    y = torch.from_numpy(oatt.rotate(g, tab, pos, interleaved, transposed=True))
    a, b = torch.from_numpy(x).requires_grad_(), torch.from_numpy(w).requires_grad_()
    (y * a * (a.square().mean(-1, keepdim=True) + eps).rsqrt() * (offset + b)).sum().backward()
    assert np.allclose(dx, a.grad.numpy(), rtol=1e-12, atol=1e-12) and np.allclose(dw, b.grad.numpy(), rtol=1e-12, atol=1e-12)

    def loss(x, w):
        return (g * norms.norm_rope(x, w, tab, pos, eps, offset, interleaved)).sum()

    h = 1e-5
    for t, i, d in [(0, 0, 0), (1, 1, 3), (2, 0, 7)]:
        e = np.zeros_like(x)
        e[t, i, d] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[t, i, d]) < 1e-7
    e = np.zeros_like(w)
    e[5] = h
    assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[5]) < 1e-7


@pytest.mark.parametrize("window,sinks,causal", [(3, 2, True), (1, 1, True), (4, 100, True), (5, 3, False), (2, 0, True)])
def test_sinks_are_a_mask(window, sinks, causal):
    r = np.random.default_rng(3)
    n, L, D = 6, 11, 16
    q, k, v = r.standard_normal((n, D)), r.standard_normal((L, D)), r.standard_normal((L, D))
    pos = list(range(L - n, L))
    o, lse, *_ = oatt.softmax_rows(q, k, v, pos, window=window, causal=causal, sinks=sinks)
    t, j = np.array(pos)[:, None], np.arange(L)[None]
    seen = ((j > t - window) | (j < sinks)) & (j <= t if causal else True)
    x = torch.from_numpy(np.where(seen, q @ k.T / math.sqrt(D), -np.inf))
    assert np.allclose(o, (torch.softmax(x, -1) @ torch.from_numpy(v)).numpy())
    assert np.allclose(lse, torch.logsumexp(x, -1).numpy())
