"""Oracle of block-scaled E4M3 quantisation, products with it in float64, and
the layer of a few tokens."""
from __future__ import annotations

import numpy as np

from . import formats


def group_codes(v):
    """(codes, scale) of one group of values: the rule's three roundings are
    binary32, the code is the nearest E4M3FN value, ties to even."""
    v = np.asarray(v, dtype=np.float32)
    a = np.float32(np.max(np.abs(v)))                # NaN if one is there
    if not np.isnan(a):
        a = np.maximum(a, np.float32(2.0 ** -100))
    with np.errstate(invalid="ignore", over="ignore"):
        q = (v * (np.float32(448) / a)).astype(np.float64)
        codes = np.where(np.isnan(q), 0x7F, formats.encode_e4m3(np.where(np.isnan(q), 0, q))).astype(np.uint8)
        return codes, a / np.float32(448)


def pad(n):
    return -(-n // 128) * 128


def quantise_rows(x):
    """codes [R, P(K)], scales [P(K)/128, R] of x [R, K]."""
    R, K = x.shape
    g = np.zeros((R, pad(K)))
    g[:, :K] = x
    codes = np.zeros(g.shape, dtype=np.uint8)
    scales = np.zeros((pad(K) // 128, R), dtype=np.float32)
    for r in range(R):
        for c in range(0, pad(K), 128):
            codes[r, c:c + 128], scales[c // 128, r] = group_codes(g[r, c:c + 128])
    return codes, scales


def quantise_blocks(w):
    """codes [N, P(K)], scales [P(N)/128, P(K)/128] of w [N, K]."""
    N, K = w.shape
    g = np.zeros((pad(N), pad(K)))
    g[:N, :K] = w
    codes = np.zeros(g.shape, dtype=np.uint8)
    scales = np.zeros((pad(N) // 128, pad(K) // 128), dtype=np.float32)
    for n in range(0, pad(N), 128):
        for c in range(0, pad(K), 128):
            q, scales[n // 128, c // 128] = group_codes(g[n:n + 128, c:c + 128].reshape(-1))
            codes[n:n + 128, c:c + 128] = q.reshape(128, 128)
    return codes[:N], scales


def values(codes):
    return formats.E4M3_TABLE[np.asarray(codes)]


def row_values(codes, scales):
    """float64 values of rows' codes [R, K] with scales [K/128, R]."""
    return values(codes) * np.repeat(scales.astype(np.float64).T, 128, axis=1)


def block_values(codes, scales):
    """float64 values of weights' codes [N, K] with scales [P(N)/128, K/128]."""
    return values(codes) * np.repeat(np.repeat(scales.astype(np.float64), 128, axis=0)[:codes.shape[0]], 128, axis=1)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def gated_backward(z, da):
    n = z.shape[1] // 2
    g, u = z[:, :n], z[:, n:]
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return np.concatenate([da * u * s * (1.0 + g * (1.0 - s)), da * g * s], axis=1)


def layer(x, router, bias, k, gate_up, down, base=None):
    """The layer on float64 weights gate_up(e) [2I, H] and down(e) [H, I]:
    (out, ids, weights, logits)."""
    z = x @ router.T + (0.0 if bias is None else bias)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    out = np.zeros_like(x) if base is None else np.array(base, dtype=np.float64)
    w = np.zeros(ids.shape)
    for t in range(x.shape[0]):
        p = np.exp(z[t, ids[t]] - z[t, ids[t, 0]])
        w[t] = p / p.sum()
        for j, e in enumerate(ids[t]):
            gu = gate_up(e) @ x[t]
            n = gu.size // 2
            out[t] += w[t, j] * (down(e) @ (silu(gu[:n]) * gu[n:]))
    return out, ids, w, z
