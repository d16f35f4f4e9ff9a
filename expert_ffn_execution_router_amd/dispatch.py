"""Expert dispatch on torch tensors: pairs sorted by expert, rows copied to
their grouped places and back with weights, and the gradients.

The caller owns every tensor; results go into tensors it passes.  ids are
int32 [T, k] with ids outside [0, E) dropped; counts, offsets, perm and pos
are what sort() writes (moe_sort in include/moe.h has their meaning).  Hidden
rows are bf16, fp16 or fp32 [rows, cols] views with contiguous rows.  Calls
enqueue on the current stream of the tensors' device (or `stream`, which the
caller orders after the work that made the inputs) and can be captured.  The
memory from a result's first to its last value must not meet an input's or
another result's, except for unpermute's base in place.  No call records a
graph: with gradients enabled, a tensor that requires grad is refused.

A forward and backward of the experts' surroundings:

    sort(ids, counts, offsets, perm, pos)
    permute(x, perm, pos, xs)                  # xs -> experts -> y
    unpermute(y, pos, w, out)
    unpermute_backward(dout, y, perm, pos, w, dy, dw)    # dy -> experts -> dxs
    permute_backward(dxs, pos, dx)
    gate_backward(ids, w, dw, dlogits)
"""
from __future__ import annotations

import torch

from . import _args as A
from . import binding as B

_I32, _F32 = torch.int32, torch.float32
_lib = B.lib


def sort_rows(T: int, k: int, E: int, align: int = 1) -> int:
    """Rows perm (and the grouped tensors) need for any routing of T tokens."""
    n = -1 if (T | k | E | align) >> 31 else B.moe_sort_rows(T, k, E, align)
    if n < 0:
        raise ValueError("need T >= 0 and k, E, align >= 1, all below 2^31")
    return n


def sort_workspace_bytes(T: int, k: int, E: int) -> int:
    if (T | k | E) >> 31:
        raise ValueError("need T >= 0 and k, E >= 1, all below 2^31")
    return B.moe_sort_workspace_bytes(T, k, E)


def sort(ids, counts, offsets, perm, pos, align=1, ws=None, stream=None):
    """Groups the pairs of ids by expert, segments padded to multiples of
    align.  ws: uint8 tensor of sort_workspace_bytes that starts on 4 bytes;
    None allocates one where it is needed (more than 2048 pairs)."""
    shape = ids.shape
    if len(shape) != 2:
        raise ValueError(f"ids: shape {tuple(shape)}, expected [T, k]")
    if align >> 31:
        raise ValueError(f"align: {align}, need 1 <= align < 2^31")
    T, k = shape
    dev, E, rows = ids.get_device(), counts.numel(), perm.numel()
    args = (A.whole("ids", ids, dev, _I32), T, k, E, align, A.whole("counts", counts, dev, _I32, (E,)),
            A.whole("offsets", offsets, dev, _I32, (E + 1,)), A.whole("perm", perm, dev, _I32, (rows,)), rows,
            A.whole("pos", pos, dev, _I32, shape))
    if ws is None:
        need = B.moe_sort_workspace_bytes(T, k, E) if T * k > 2048 else 0
        if need and dev >= 0:
            if stream is None:
                ws = torch.empty(need, dtype=torch.uint8, device=ids.device)
            else:
                with torch.cuda.stream(stream):
                    ws = torch.empty(need, dtype=torch.uint8, device=ids.device)
    wp, wn = (None, 0) if ws is None else (A.whole("ws", ws, dev, torch.uint8), ws.numel())
    A.launch(_lib().moe_sort, dev, stream, *args, wp, wn)


def _tokens(name, pos, dev):
    shape = pos.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [T, k]")
    return A.whole(name, pos, dev, _I32), shape


def permute(x, perm, pos, out, stream=None):
    """out[pos[t, j]] = x[t]; rows with perm -1 become zero, rows behind the
    last segment stay.  perm None: no padding rows (align 1)."""
    dev, cols, n = x.get_device(), x.shape[-1], out.shape[0]
    pp, (T, k) = _tokens("pos", pos, dev)
    dt, xp, ldx, xe = A.rows("x", x, dev, T, cols)
    ot, op, ldo, oe = A.rows("out", out, dev, n, cols)
    if ot != dt:
        raise ValueError(f"out: type {out.dtype}, x has {x.dtype}")
    if xp < oe and op < xe:
        A.overlaps("out")
    rp = None if perm is None else A.whole("perm", perm, dev, _I32, (n,))
    A.launch(_lib().moe_permute, dev, stream, dt, xp, ldx, rp, pp, T, k, n, cols, op, ldo)


def unpermute(y, pos, w, out, base=None, stream=None):
    """out[t] = base[t] + sum_j w[t, j] y[pos[t, j]] over the kept pairs, summed
    in fp32.  w: fp32 [T, k] or None for ones; base: fp32 [T, cols] or None.
    y and out: one type, or one of them fp32."""
    dev, cols, n = y.get_device(), y.shape[-1], y.shape[0]
    pp, shape = _tokens("pos", pos, dev)
    T, k = shape
    yt, yp, ldy, ye = A.rows("y", y, dev, n, cols)
    ot, op, ldo, oe = A.rows("out", out, dev, T, cols)
    if yp < oe and op < ye:
        A.overlaps("out")
    wp = None if w is None else A.whole("w", w, dev, _F32, shape)
    bp, ldb = None, 0
    if base is not None:
        _, bp, ldb, be = A.rows("base", base, dev, T, cols, A.F32_ONLY)
        if bp < oe and op < be and (bp != op or ldb != ldo or ot != B.MOE_T_F32):       # else in place
            A.overlaps("out")
    A.launch(_lib().moe_unpermute, dev, stream, yt, yp, ldy, n, pp, wp, bp, ldb, T, k, cols, ot, op, ldo)


def permute_backward(dout, pos, dx, stream=None):
    """Gradient of permute: dx[t] = sum_j dout[pos[t, j]]."""
    unpermute(dout, pos, None, dx, stream=stream)


def unpermute_backward(dout, y, perm, pos, w, dy, dw, stream=None):
    """Gradients of unpermute: dy[pos[t, j]] = w[t, j] dout[t] and dw[t, j] =
    <dout[t], y[pos[t, j]]> (0 for dropped pairs).  Padding rows of dy become
    zero (perm None: there are none), rows behind the last segment stay.  After
an unpermute without weights dy is permute(dout)."""
    dev, cols, n = y.get_device(), y.shape[-1], y.shape[0]
    pp, shape = _tokens("pos", pos, dev)
    T, k = shape
    yt, yp, ldy, ye = A.rows("y", y, dev, n, cols)
    ot, gp, ldd, ge = A.rows("dout", dout, dev, T, cols)
    dt, dp, lddy, de = A.rows("dy", dy, dev, n, cols)
    if dt != yt:
        raise ValueError(f"dy: type {dy.dtype}, y has {y.dtype}")
    if (yp < de and dp < ye) or (gp < de and dp < ge):
        A.overlaps("dy")
    rp = None if perm is None else A.whole("perm", perm, dev, _I32, (n,))
    A.launch(_lib().moe_unpermute_backward, dev, stream, ot, gp, ldd, yt, yp, ldy, rp, n, pp,
             A.whole("w", w, dev, _F32, shape), T, k, cols, dp, lddy, A.whole("dw", dw, dev, _F32, shape))


def gate_backward(ids, w, dw, dlogits, stream=None):
    """Gradient of the softmax over the chosen logits: dlogits fp32 [T, E],
    zero where an expert was not chosen."""
    dev, E = ids.get_device(), dlogits.shape[-1]
    ip, shape = _tokens("ids", ids, dev)
    T, k = shape
    _, zp, ldz, ze = A.rows("dlogits", dlogits, dev, T, E, A.F32_ONLY)
    wp, dp, size = A.whole("w", w, dev, _F32, shape), A.whole("dw", dw, dev, _F32, shape), 4 * T * k
    if (wp < ze and zp < wp + size) or (dp < ze and zp < dp + size):
        A.overlaps("dlogits")
    A.launch(_lib().moe_gate_backward, dev, stream, ip, wp, dp, T, k, E, zp, ldz)
