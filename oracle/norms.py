"""Float64 oracle of the norms around a block and their gradients, written from
the formulas (the gradients through each row's Jacobian)."""
from __future__ import annotations

import numpy as np


def rms(v, eps):
    return np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def before(r, w, eps):
    return r / rms(r, eps) * w


def after(y, r, alpha, w, gate, eps):
    """out: y [T, n]; w None: y as it is; gate None: ones; r None: zero."""
    v = y if w is None else y / rms(y, eps) * w
    if gate is not None:
        v = gate * v
    return v if r is None else alpha * r + v


def through_rms(v, d, eps):
    """d^T of the Jacobian of v / rms(v), row by row: I / rms - v v^T / (n rms^3)."""
    out = np.empty_like(v)
    n = v.shape[1]
    for t in range(v.shape[0]):
        s = np.sqrt(np.mean(v[t] ** 2) + eps)
        out[t] = d[t] / s - v[t] * np.dot(v[t], d[t]) / (n * s ** 3)
    return out


def backward(dout, dnext, y, h, alpha, w, gate, w2, eps, eps2):
    """Gradients of out = after(...) and next = before(h = out): (dy, dr, dw,
    dgate, dw2); None where there is none."""
    d = np.zeros_like(h if dout is None else dout) if dout is None else np.array(dout)
    dw2 = None
    if dnext is not None:
        d = d + through_rms(h, dnext * w2, eps2)
        dw2 = np.sum(dnext * h / rms(h, eps2), axis=0)
    if y is None:
        return None, alpha * d, None, None, dw2
    g = np.ones((1, 1)) if gate is None else gate
    x = y if w is None else y / rms(y, eps)
    v = x if w is None else x * w
    dgate = None
    if gate is not None:
        dgate = d * v
        for axis in (0, 1):
            if gate.shape[axis] == 1 and dgate.shape[axis] != 1:
                dgate = dgate.sum(axis, keepdims=True)
    dv = d * g
    dw = None if w is None else np.sum(dv * x, axis=0)
    dy = dv if w is None else through_rms(y, dv * w, eps)
    return dy, alpha * d, dw, dgate, dw2
