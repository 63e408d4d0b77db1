"""NumPy values of a key/value cache of 8 bits: rounding to e4m3, the scale of a block,
and the append, one block at a time.  Test infrastructure only.
"""

from __future__ import annotations

import math

import numpy as np

MOST, LEAST_SCALE = 448.0, 2.0 ** -100


def e4m3(x) -> np.ndarray:
    """Nearest e4m3 value, ties to even: 3 fraction bits from 2^-6 on, steps of 2^-9 below."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
        step = 2.0 ** (e - 3)
        return np.where(np.isfinite(x), np.round(x / step) * step, np.nan)


def scale_of(top: float) -> float:
    """The least power of two with which ``top`` is at most 448."""
    if top <= 0:
        return LEAST_SCALE
    s = 2.0 ** math.ceil(math.log2(top / MOST))
    while top / s > MOST:
        s *= 2
    while top / (s / 2) <= MOST:
        s /= 2
    return max(s, LEAST_SCALE)


def append(cache, scale, rows, new, lengths, page_indices, page_indptr, page_size: int, block: int, most=None):
    """Writes rows [T, H, D] (the last new[b] of lengths[b] tokens of each sequence) to codes ``cache``
    [pages, page_size, H, D] and ``scale`` [pages, blocks, H], fp64 arrays changed in place.  ``most``: the largest
    magnitude that is stored."""
    t = 0
    for b, n in enumerate(new):
        first = lengths[b] - n  # position of the first new token
        for lo in range(first // block * block, lengths[b], block):
            a, z = max(lo, first, 0), min(lo + block, lengths[b])
            if z <= a:
                continue
            page = int(page_indices[int(page_indptr[b]) + lo // page_size])
            sub, off = lo % page_size // block, lo % page_size
            x = np.array(rows[t + a - first:t + z - first], dtype=np.float64)
            x[~np.isfinite(x)] = np.nan
            if most:
                x = np.clip(x, -most, most)
            for h in range(x.shape[1]):
                top = np.nanmax(np.abs(x[:, h])) if np.isfinite(x[:, h]).any() else 0.0
                s = scale_of(top)
                if a > lo:
                    old = scale[page, sub, h]
                    s = max(s, old)
                    if s > old:
                        kept = cache[page, off:off + a - lo, h]
                        cache[page, off:off + a - lo, h] = e4m3(kept * (old / s))
                cache[page, off + a - lo:off + z - lo, h] = e4m3(x[:, h] / s)
                scale[page, sub, h] = s
        t += n
