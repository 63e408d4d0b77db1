"""fp64 NumPy values of the attention layers' operators: the rotary table and
map, the append to a paged cache, and attention over it, each written straight
from its definition, one row at a time.  Test infrastructure only.
"""

from __future__ import annotations

import math
from typing import Optional

import numpy as np


def frequencies(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                original: float = 0.0, low_turns: float = 1.0, high_turns: float = 4.0) -> np.ndarray:
    """Angle per token of each of the rot / 2 pairs."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        turns = original * f / (2 * math.pi)
        w = np.clip((turns - low_turns) / (high_turns - low_turns), 0.0, 1.0)
        return f * ((1 - w) / factor + w)
    return f


def table(positions: int, rot: int, magnitude: float = 1.0, **kw) -> np.ndarray:
    """[positions, rot]: cosines, then sines."""
    a = np.arange(positions, dtype=np.float64)[:, None] * frequencies(rot, **kw)
    return magnitude * np.concatenate([np.cos(a), np.sin(a)], axis=1)


def rotate(x: np.ndarray, tab: np.ndarray, positions, interleaved: bool = False,
           transposed: bool = False) -> np.ndarray:
    """x [T, H, D] turned pair by pair with rows ``positions`` of ``tab`` [P, rot]."""
    y = np.array(x, dtype=np.float64)
    r = tab.shape[1]
    for t, pos in enumerate(positions):
        c, s = tab[pos, :r // 2].astype(np.float64), tab[pos, r // 2:].astype(np.float64)
        if transposed:
            s = -s
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
            u, w = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a] = u * c[i] - w * s[i]
            y[t, :, b] = w * c[i] + u * s[i]
    return y


def slots(page_indices, page_indptr, last_page_len, page_size: int, b: int):
    """(page, offset) of every token sequence b holds, in order."""
    first, end = int(page_indptr[b]), int(page_indptr[b + 1])
    n = (end - first - 1) * page_size + int(last_page_len[b]) if end > first else 0
    return [(int(page_indices[first + j // page_size]), j % page_size) for j in range(n)]


def softmax_rows(q: np.ndarray, k: np.ndarray, v: np.ndarray, positions, scale: Optional[float] = None,
                 softcap: float = 0.0, window: int = 0, causal: bool = True):
    """q [n, D] at ``positions`` against k, v [L, D]: (o [n, D], lse [n], magnitude [n, D] =
    sum p |v|, spread [n] = largest sum |q_d k_d| times the scale, reach [n] = largest |x|)."""
    n, D = q.shape
    L = k.shape[0]
    scale = scale or 1.0 / math.sqrt(D)
    o, mag = np.zeros((n, D)), np.zeros((n, D))
    lse, spread, reach = np.full(n, -np.inf), np.zeros(n), np.zeros(n)
    for i, t in enumerate(positions):
        lo = max(0, t - window + 1) if window else 0
        hi = min(t, L - 1) if causal else L - 1
        if hi < lo:
            continue
        kk, vv = k[lo:hi + 1], v[lo:hi + 1]
        x = scale * (kk @ q[i])
        if softcap:
            x = softcap * np.tanh(x / softcap)
        top = x.max()
        e = np.exp(x - top)
        p = e / e.sum()
        o[i], mag[i] = p @ vv, p @ np.abs(vv)
        lse[i] = top + math.log(e.sum())
        spread[i] = scale * (np.abs(kk) @ np.abs(q[i])).max()
        reach[i] = np.abs(x).max()
    return o, lse, mag, spread, reach


def attention_paged(q, cu_seqlens, k_cache, v_cache, page_indices, page_indptr, page_size, last_page_len,
                    scale=None, softcap=0.0, window=0, causal=True):
    """The five arrays of softmax_rows for q [T, Hq, D], caches [pages, page_size, Hkv, D].
    Only slots that a sequence holds are read."""
    T, Hq, D = q.shape
    Hk = k_cache.shape[2]
    G = Hq // Hk
    o, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, spread, reach = np.full((T, Hq), -np.inf), np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(last_page_len)):
        t0, t1 = (b, b + 1) if cu_seqlens is None else (int(cu_seqlens[b]), int(cu_seqlens[b + 1]))
        where = slots(page_indices, page_indptr, last_page_len, page_size, b)
        if t1 == t0 or not where:
            continue
        pg, off = np.array([w[0] for w in where]), np.array([w[1] for w in where])
        pos = [len(where) - (t1 - t0) + i for i in range(t1 - t0)]
        for h in range(Hk):
            k = np.asarray(k_cache[pg, off, h], dtype=np.float64)
            v = np.asarray(v_cache[pg, off, h], dtype=np.float64)
            for g in range(G):
                got = softmax_rows(np.asarray(q[t0:t1, h * G + g], dtype=np.float64), k, v, pos, scale, softcap,
                                   window, causal)
                for dst, x in zip((o, lse, mag, spread, reach), got):
                    dst[t0:t1, h * G + g] = x
    return o, lse, mag, spread, reach
