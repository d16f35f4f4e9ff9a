"""Float64 oracle of expert dispatch: pairs sorted by expert, rows to their
grouped places and back, and the gradients.  Plain loops and index sums."""
from __future__ import annotations

import numpy as np


def sort_pairs(ids: np.ndarray, E: int, align: int, rows: int):
    """(counts, offsets, perm, pos) of int ids [T, k]; see the arguments of
    the library's sort."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    groups = [[] for _ in range(E)]
    for a, e in enumerate(flat):
        if 0 <= e < E:
            groups[e].append(a)
    counts = np.array([len(g) for g in groups], dtype=np.int32)
    offsets = np.zeros(E + 1, dtype=np.int32)
    perm = np.full(rows, -2, dtype=np.int32)
    pos = np.full(T * k, -1, dtype=np.int32)
    at = 0
    for e, g in enumerate(groups):
        offsets[e] = at
        size = -(-len(g) // align) * align
        perm[at:at + size] = -1
        perm[at:at + len(g)] = g
        pos[g] = np.arange(at, at + len(g))
        at += size
    offsets[E] = at
    return counts, offsets, perm, pos.reshape(T, k)


def permute(x, perm, pos, out):
    """out (rows before the call) with token rows and zeroed padding."""
    out = np.array(out)
    out[np.nonzero(perm == -1)[0]] = 0
    T, k = pos.shape
    for j in range(k):
        t = np.nonzero(pos[:, j] >= 0)[0]
        out[pos[t, j]] = x[t]
    return out


def unpermute(y, pos, w, base, cols):
    """(out, magnitude): the sum and the sum of the terms' absolute values."""
    T, k = pos.shape
    out = np.zeros((T, cols)) if base is None else np.array(base, dtype=np.float64)
    mag = np.abs(out)
    for j in range(k):
        t = np.nonzero(pos[:, j] >= 0)[0]
        term = y[pos[t, j]] * (1.0 if w is None else w[t, j][:, None])
        out[t] += term
        mag[t] += np.abs(term)
    return out, mag


def unpermute_backward(dout, y, perm, pos, w, dy):
    """(dy, dw, magnitude of dw's sums); dy's rows behind the segments kept."""
    dy = np.array(dy, dtype=np.float64)
    dy[np.nonzero(perm == -1)[0]] = 0
    dw = np.zeros(pos.shape)
    mag = np.zeros(pos.shape)
    for j in range(pos.shape[1]):
        t = np.nonzero(pos[:, j] >= 0)[0]
        r = pos[t, j]
        dy[r] = w[t, j][:, None] * dout[t]
        dw[t, j] = (dout[t] * y[r]).sum(1)
        mag[t, j] = np.abs(dout[t] * y[r]).sum(1)
    return dy, dw, mag


def gate_backward(ids, w, dw, E):
    """(dz, magnitude) through the softmax over each token's chosen logits."""
    T, k = ids.shape
    inner, imag = (w * dw).sum(1, keepdims=True), np.abs(w * dw).sum(1, keepdims=True)
    g, gm = w * (dw - inner), w * (np.abs(dw) + imag)
    dz, mag = np.zeros((T, E)), np.zeros((T, E))
    for j in range(k):
        t = np.nonzero((ids[:, j] >= 0) & (ids[:, j] < E))[0]
        dz[t, ids[t, j]] += g[t, j]
        mag[t, ids[t, j]] += gm[t, j]
    return dz, mag
