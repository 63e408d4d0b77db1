"""fp64 NumPy values of the norm of query and key heads before the rotation, and of its
gradient, from the definition.  Test infrastructure only.
"""

from __future__ import annotations

import numpy as np

from .attention import rotate


def norm_rope(x: np.ndarray, w: np.ndarray, tab: np.ndarray, positions, eps: float, offset: float = 0.0,
              interleaved: bool = False) -> np.ndarray:
    """x [T, H, D] normed with w [D], then turned with rows ``positions`` of ``tab``."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * (offset + np.asarray(w, dtype=np.float64))
    return rotate(y, tab, positions, interleaved)


def norm_rope_grad(g: np.ndarray, x: np.ndarray, w: np.ndarray, tab: np.ndarray, positions, eps: float,
                   offset: float = 0.0, interleaved: bool = False):
    """(dx, dw) for the gradient g of norm_rope's output: with m = mean x^2 + eps, y = R^T g and
    n = y (offset + w), d(x_j m^(-1/2))/dx_i = m^(-1/2) (delta_ij - x_i x_j / (D m))."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    m = (x * x).mean(axis=-1, keepdims=True) + eps
    y = rotate(g, tab, positions, interleaved, transposed=True)
    n = y * (offset + w)
    dx = (n - x * (n * x).mean(axis=-1, keepdims=True) / m) / np.sqrt(m)
    return dx, (y * x / np.sqrt(m)).sum(axis=(0, 1))
