"""Float64 oracle of products with 4-bit weights and group scales."""
from __future__ import annotations

import numpy as np


def pack(q: np.ndarray) -> np.ndarray:
    """Codes 0..15 [..., K] to bytes [..., K/2], even input in the low nibble."""
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def dequantise(q, scales, zeros, group):
    """float64 weights of codes q [N, K]; zeros None: 8."""
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, axis=-1)
    return (q.astype(np.float64) - z) * np.repeat(scales.astype(np.float64), group, axis=-1)


def product(x, q, scales, zeros, group):
    """(z, magnitude): x W^T and the sum of |x| (q + |zero|) |scale|, which
    bounds every partial sum of either side of q - zero."""
    w = dequantise(q, scales, zeros, group)
    z8 = 8.0 if zeros is None else np.repeat(np.abs(zeros.astype(np.float64)), group, axis=-1)
    m = (q.astype(np.float64) + z8) * np.repeat(np.abs(scales.astype(np.float64)), group, axis=-1)
    return x @ w.T, np.abs(x) @ m.T


def silu(g):
    return g / (1.0 + np.exp(-g))
