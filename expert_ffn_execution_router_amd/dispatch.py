"""Expert dispatch on torch tensors: pairs sorted by expert, rows copied to
their grouped places and back with weights, and the gradients.

The caller owns every tensor; results go into tensors it passes.  ids are
int32 [T, k] with ids outside [0, E) dropped; counts, offsets, perm and pos
are what sort() writes (moe_sort in include/moe.h has their meaning).  Hidden
rows are bf16, fp16 or fp32 [rows, cols] views with contiguous rows.  Calls
enqueue on the current stream of the tensors' device (or `stream`, which the
caller orders after the work that made the inputs) and can be captured.

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


def sort_rows(T: int, k: int, E: int, align: int = 1) -> int:
    """Rows perm (and the grouped tensors) need for any routing of T tokens."""
    n = B.moe_sort_rows(T, k, E, align)
    if n < 0:
        raise ValueError("need T >= 0 and k, E, align >= 1")
    return n


def sort_workspace_bytes(T: int, k: int, E: int) -> int:
    return B.moe_sort_workspace_bytes(T, k, E)


def sort(ids, counts, offsets, perm, pos, align=1, ws=None, stream=None):
    """Groups the pairs of ids by expert, segments padded to multiples of
    align.  ws: uint8 tensor of sort_workspace_bytes; None allocates one where
    it is needed (more than 2048 pairs)."""
    if ids.dim() != 2:
        raise ValueError(f"ids: shape {tuple(ids.shape)}, expected [T, k]")
    T, k = ids.shape
    dev, E = ids.device, counts.numel()
    i32 = torch.int32
    need = B.moe_sort_workspace_bytes(T, k, E)
    if need and ws is None:
        if stream is None:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(stream):
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
    wp, wn = (None, 0) if ws is None else (A.whole("ws", ws, dev, torch.uint8, (ws.numel(),)), ws.numel())
    rows = perm.numel()
    A.launch(B.moe_sort, dev, stream, A.whole("ids", ids, dev, i32, (T, k)), T, k, E, align,
             A.whole("counts", counts, dev, i32, (E,)), A.whole("offsets", offsets, dev, i32, (E + 1,)),
             A.whole("perm", perm, dev, i32, (rows,)), rows, A.whole("pos", pos, dev, i32, (T, k)), wp, wn)


def _pos(pos, dev):
    if pos.dim() != 2:
        raise ValueError(f"pos: shape {tuple(pos.shape)}, expected [T, k]")
    T, k = pos.shape
    return A.whole("pos", pos, dev, torch.int32, (T, k)), T, k


def permute(x, perm, pos, out, stream=None):
    """out[pos[t, j]] = x[t]; rows with perm -1 become zero, rows behind the
    last segment stay.  perm None: no padding rows (align 1)."""
    dev = x.device
    pp, T, k = _pos(pos, dev)
    dt, ldx = A.rows("x", x, dev)
    if x.shape[0] != T:
        raise ValueError(f"x: {x.shape[0]} rows, pos has {T} tokens")
    if out.dtype != x.dtype:
        raise ValueError(f"out: type {out.dtype}, x has {x.dtype}")
    _, ldo = A.rows("out", out, dev, x.shape[1])
    A.apart("out", out, x)
    rows = out.shape[0]
    rp = None if perm is None else A.whole("perm", perm, dev, torch.int32, (rows,))
    A.launch(B.moe_permute, dev, stream, dt, x.data_ptr(), ldx, rp, pp, T, k, rows, x.shape[1], out.data_ptr(), ldo)


def unpermute(y, pos, w, out, base=None, stream=None):
    """out[t] = base[t] + sum_j w[t, j] y[pos[t, j]] over the kept pairs, summed
    in fp32.  w: fp32 [T, k] or None for ones; base: fp32 [T, cols] or None.
    y and out: one type, or one of them fp32."""
    dev = y.device
    pp, T, k = _pos(pos, dev)
    yt, ldy = A.rows("y", y, dev)
    cols = y.shape[1]
    ot, ldo = A.rows("out", out, dev, cols)
    if out.shape[0] != T:
        raise ValueError(f"out: {out.shape[0]} rows, pos has {T} tokens")
    A.apart("out", out, y)
    wp = None if w is None else A.whole("w", w, dev, torch.float32, (T, k))
    bp, ldb = None, 0
    if base is not None:
        _, ldb = A.rows("base", base, dev, cols, {torch.float32: B.MOE_T_F32})
        if base.shape[0] != T:
            raise ValueError(f"base: {base.shape[0]} rows, pos has {T} tokens")
        bp = base.data_ptr()
        if bp != out.data_ptr() or ldb != ldo or out.dtype != torch.float32:
            A.apart("out", out, base)
    A.launch(B.moe_unpermute, dev, stream, yt, y.data_ptr(), ldy, y.shape[0], pp, wp, bp, ldb, T, k, cols, ot,
             out.data_ptr(), ldo)


def permute_backward(dout, pos, dx, stream=None):
    """Gradient of permute: dx[t] = sum_j dout[pos[t, j]]."""
    unpermute(dout, pos, None, dx, stream=stream)


def unpermute_backward(dout, y, perm, pos, w, dy, dw, stream=None):
    """Gradients of unpermute: dy[pos[t, j]] = w[t, j] dout[t] and dw[t, j] =
    <dout[t], y[pos[t, j]]> (0 for dropped pairs).  Padding rows of dy become
    zero (perm None: there are none), rows behind the last segment stay."""
    dev = y.device
    pp, T, k = _pos(pos, dev)
    yt, ldy = A.rows("y", y, dev)
    rows, cols = y.shape
    ot, ldd = A.rows("dout", dout, dev, cols)
    if dout.shape[0] != T:
        raise ValueError(f"dout: {dout.shape[0]} rows, pos has {T} tokens")
    if dy.dtype != y.dtype or dy.shape != y.shape:
        raise ValueError(f"dy: {dy.dtype} {tuple(dy.shape)}, y is {y.dtype} {tuple(y.shape)}")
    _, lddy = A.rows("dy", dy, dev, cols)
    A.apart("dy", dy, y, dout)
    rp = None if perm is None else A.whole("perm", perm, dev, torch.int32, (rows,))
    A.launch(B.moe_unpermute_backward, dev, stream, ot, dout.data_ptr(), ldd, yt, y.data_ptr(), ldy, rp, rows, pp,
             A.whole("w", w, dev, torch.float32, (T, k)), T, k, cols, dy.data_ptr(), lddy,
             A.whole("dw", dw, dev, torch.float32, (T, k)))


def gate_backward(ids, w, dw, dlogits, stream=None):
    """Gradient of the softmax over the chosen logits: dlogits fp32 [T, E],
    zero where an expert was not chosen."""
    dev = ids.device
    if ids.dim() != 2:
        raise ValueError(f"ids: shape {tuple(ids.shape)}, expected [T, k]")
    T, k = ids.shape
    _, ldz = A.rows("dlogits", dlogits, dev, None, {torch.float32: B.MOE_T_F32})
    if dlogits.shape[0] != T:
        raise ValueError(f"dlogits: {dlogits.shape[0]} rows, ids has {T} tokens")
    A.apart("dlogits", dlogits, w, dw)
    A.launch(B.moe_gate_backward, dev, stream, A.whole("ids", ids, dev, torch.int32, (T, k)),
             A.whole("w", w, dev, torch.float32, (T, k)), A.whole("dw", dw, dev, torch.float32, (T, k)), T, k,
             dlogits.shape[1], dlogits.data_ptr(), ldz)
