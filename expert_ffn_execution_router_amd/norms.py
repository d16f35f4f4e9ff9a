"""The norms before and after a block on torch tensors, fused with the block's
gate and residual scale, and their gradients:

    before   next = (r / rms(r)) w2
    after    out  = alpha r + gate * (y / rms(y)) w
             next = (out / rms(out)) w2

with rms(v) = sqrt(mean v^2 + eps) over a row of up to 16384 columns (8192 for
the gradients).  y (the
block's result) and next have one type, the residual rows r and out that type
or fp32; weights [cols] and the gate ([T, 1], [1, cols] or [T, cols]) y's type
or fp32.  next may be e4m3 codes [T, padded(cols)] with scales
[padded(cols)/128, T] as fp8.quantize gives them.  out is rounded once; the next
norm is that of the rounded rows.

The caller owns every tensor; results go into tensors it passes.  Calls enqueue
on the current stream of the tensors' device (or `stream`, which the caller
orders after the work that made the inputs) and can be captured.  A result's
memory must not meet an input's or another result's, except that out may be the
residual itself.  No call records a graph: with gradients enabled, a tensor
that requires grad is refused.  moe_norm and moe_norm_backward in
include/moe.h have the details.
"""
from __future__ import annotations

import torch

from . import _args as A
from . import binding as B

_F32, F8 = torch.float32, torch.float8_e4m3fn
# types of what goes with rows of a type: that type or fp32
_WITH = {dt: {dt: code, _F32: B.MOE_T_F32} for dt, code in A.TYPES.items()}


def _weight(name, w, dev, cols, types):
    """Type code and address of a weight."""
    code = types.get(w.dtype)
    if code is None:
        raise ValueError(f"{name}: type {w.dtype} is not one of {[str(x) for x in types]}")
    return code, A.whole(name, w, dev, w.dtype, (cols,))


def _weights(weight, next_weight, dev, cols, types):
    """Their one type code and addresses (None: not there)."""
    if weight is None:
        if next_weight is None:
            return B.MOE_T_F32, None, None
        code, p = _weight("next_weight", next_weight, dev, cols, types)
        return code, None, p
    code, p = _weight("weight", weight, dev, cols, types)
    if next_weight is None:
        return code, p, None
    other, q = _weight("next_weight", next_weight, dev, cols, types)
    if other != code:
        raise ValueError(f"next_weight: type {next_weight.dtype}, weight has {weight.dtype}")
    return code, p, q


def _gate(name, g, dev, T, cols, types):
    """Type code, address and strides (0 along a spread axis)."""
    if g is None:
        return B.MOE_T_F32, None, 0, 0
    shape = tuple(g.shape)
    if shape not in ((T, 1), (1, cols), (T, cols)):
        raise ValueError(f"{name}: shape {shape}, expected [{T}, 1], [1, {cols}] or [{T}, {cols}]")
    code, p, ld, _ = A.rows(name, g, dev, None, shape[1], types)
    if shape == (T, 1):
        return code, p, ld, 0
    return code, p, 0 if shape[0] == 1 else ld, 1


def _next(name, out, scales, dev, T, cols, dtype):
    """Address, row stride and scales' address of the next norm's rows."""
    if out.dtype != F8:
        if scales is not None:
            raise ValueError(f"{name}: scales belong to e4m3 codes, type {out.dtype}")
        code, p, ld, _ = A.rows(name, out, dev, T, cols)
        if code != A.TYPES[dtype]:
            raise ValueError(f"{name}: type {out.dtype}, expected {dtype}")
        return p, ld, None
    if scales is None:
        raise ValueError(f"{name}: e4m3 codes need scales")
    width = (cols + 127) // 128 * 128
    return (A.whole(name, out, dev, F8, (T, width)), width,
            A.whole(f"{name} scales", scales, dev, _F32, (width // 128, T)))


def _block_type(name, t):
    if t.dtype not in A.TYPES:
        raise ValueError(f"{name}: type {t.dtype} is not one of {[str(x) for x in A.TYPES]}")
    return t.dtype


def before(x, weight, out, scales=None, eps=1e-6, stream=None):
    """out = (x / rms(x)) weight.  out: x's type, a 16-bit type where x is fp32,
    or e4m3 codes with scales."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected rows")
    dev, (T, cols) = x.get_device(), x.shape
    _block_type("x", x)
    # the block's type: that of the rows it reads
    dtype = out.dtype if out.dtype != F8 else weight.dtype if weight.dtype != _F32 else x.dtype
    if dtype not in _WITH:
        raise ValueError(f"out: type {dtype} is not one of {[str(x) for x in A.TYPES]}")
    types = _WITH[dtype]
    rt, xp, ldx, _ = A.rows("x", x, dev, T, cols, types)
    wt, wp = _weight("weight", weight, dev, cols, types)
    op, ldo, sp = _next("out", out, scales, dev, T, cols, dtype)
    A.launch(B.lib().moe_norm, dev, stream, A.TYPES[dtype], None, 0, rt, xp, ldx, 1.0, wt, None, wt, None, 0, 0, None,
             0, wp, op, ldo, sp, T, cols, eps, eps)


def after(y, residual, out, weight=None, gate=None, alpha=1.0, eps=1e-6, next_weight=None, next_out=None,
          next_scales=None, next_eps=None, stream=None):
    """out = alpha residual + gate * (y / rms(y)) weight, and with next_out the
    next block's norm of it (next_eps None: eps).  weight None: y as it is;
    gate None: ones."""
    if y.dim() != 2:
        raise ValueError(f"y: shape {tuple(y.shape)}, expected rows")
    dev, (T, cols), dtype = y.get_device(), y.shape, _block_type("y", y)
    dt, yp, ldy, _ = A.rows("y", y, dev, T, cols)
    types = _WITH[dtype]
    rt, rp, ldr, _ = A.rows("residual", residual, dev, T, cols, types)
    ot, op, ldo, _ = A.rows("out", out, dev, T, cols, types)
    if ot != rt:
        raise ValueError(f"out: type {out.dtype}, the residual has {residual.dtype}")
    wt, wp, np_ = _weights(weight, next_weight, dev, cols, types)
    gt, gp, gr, gc = _gate("gate", gate, dev, T, cols, types)
    xp, ldx, sp = None, 0, None
    if next_out is not None:
        if next_weight is None:
            raise ValueError("next_out: needs next_weight")
        xp, ldx, sp = _next("next_out", next_out, next_scales, dev, T, cols, dtype)
    A.launch(B.lib().moe_norm, dev, stream, dt, yp, ldy, rt, rp, ldr, alpha, wt, wp, gt, gp, gr, gc, op, ldo, np_, xp,
             ldx, sp, T, cols, eps, eps if next_eps is None else next_eps)


def backward_workspace_bytes(T: int, cols: int) -> int:
    return B.moe_norm_backward_workspace_bytes(T, cols)


def _workspace(ws, T, cols, x, wanted, stream):
    return A.workspace(ws, B.moe_norm_backward_workspace_bytes(T, cols) if ws is None and wanted else 0, x, stream)


def before_backward(dout, x, weight, dx, dweight=None, base=None, eps=1e-6, ws=None, stream=None):
    """Gradients of before(): dx = base + the gradient through the norm (base:
    the residual's own, x's type), dweight fp32 [cols].  ws: uint8 tensor of
    backward_workspace_bytes, None allocates one where it is needed."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected rows")
    dev, (T, cols), dtype = x.get_device(), x.shape, _block_type("dout", dout)
    dt, gp, ldg, _ = A.rows("dout", dout, dev, T, cols)
    types = _WITH[dtype]
    rt, xp, ldx, _ = A.rows("x", x, dev, T, cols, types)
    ot, op, ldo, _ = A.rows("dx", dx, dev, T, cols, types)
    bt, bp, ldb = rt, None, 0
    if base is not None:
        bt, bp, ldb, _ = A.rows("base", base, dev, T, cols, types)
    if ot != rt or bt != rt:
        raise ValueError(f"dx and base have x's type {x.dtype}")
    wt, wp = _weight("weight", weight, dev, cols, types)
    dwp = None if dweight is None else A.whole("dweight", dweight, dev, _F32, (cols,))
    sp, sn = _workspace(ws, T, cols, x, dweight is not None, stream)
    A.launch(B.lib().moe_norm_backward, dev, stream, dt, rt, bp, ldb, None, 0, 1.0, wt, None, dt, None, 0, 0, gp, ldg,
             xp, ldx, wp, None, 0, op, ldo, None, dt, None, 0, 0, dwp, T, cols, eps, eps, sp, sn)


def after_backward(dout, y, dy, dresidual=None, weight=None, dweight=None, gate=None, dgate=None, alpha=1.0, eps=1e-6,
                   dnext=None, out=None, next_weight=None, dnext_weight=None, next_eps=None, ws=None, stream=None):
    """Gradients of after(): dout (the residual's type) that of out, dnext (y's
    type) that of next_out, either may be None; with dnext also out as after()
    wrote it and next_weight.  Written: dy (y's type), dresidual (the
    residual's type), dweight and dnext_weight (fp32 [cols]), dgate (the
    gate's shape, y's type or fp32).  ws as in before_backward."""
    if y.dim() != 2:
        raise ValueError(f"y: shape {tuple(y.shape)}, expected rows")
    dev, (T, cols), dtype = y.get_device(), y.shape, _block_type("y", y)
    dt, yp, ldy, _ = A.rows("y", y, dev, T, cols)
    types, rt = _WITH[dtype], None

    def residual(name, t):
        nonlocal rt
        if t is None:
            return None, 0
        code, p, ld, _ = A.rows(name, t, dev, T, cols, types)
        if rt is not None and code != rt:
            raise ValueError(f"{name}: type {t.dtype}, other residual rows have another")
        rt = code
        return p, ld
    if dout is None and dnext is None:
        raise ValueError("dout or dnext is needed")
    op, ldo = residual("dout", dout)
    rp, ldr = residual("dresidual", dresidual)
    hp, ldh, np_, ldn = None, 0, None, 0
    if dnext is not None:
        if out is None or next_weight is None:
            raise ValueError("dnext: needs out and next_weight")
        hp, ldh = residual("out", out)
        nt, np_, ldn, _ = A.rows("dnext", dnext, dev, T, cols)
        if nt != dt:
            raise ValueError(f"dnext: type {dnext.dtype}, y has {y.dtype}")
    dyt, dyp, lddy, _ = A.rows("dy", dy, dev, T, cols)
    if dyt != dt:
        raise ValueError(f"dy: type {dy.dtype}, y has {y.dtype}")
    wt, wp, w2p = _weights(weight, next_weight, dev, cols, types)
    gt, gp, gr, gc = _gate("gate", gate, dev, T, cols, types)
    dgt, dgp, dgr, dgc = dt, None, 0, 0
    if dgate is not None:
        if gate is None or dgate.shape != gate.shape:
            raise ValueError(f"dgate: shape {tuple(dgate.shape)}, expected the gate's")
        dgt, dgp, dgr, dgc = _gate("dgate", dgate, dev, T, cols, types)
    dwp = None if dweight is None else A.whole("dweight", dweight, dev, _F32, (cols,))
    dw2 = None if dnext_weight is None else A.whole("dnext_weight", dnext_weight, dev, _F32, (cols,))
    sums = dweight is not None or dnext_weight is not None or (dgate is not None and dgr == 0)
    sp, sn = _workspace(ws, T, cols, y, sums, stream)
    A.launch(B.lib().moe_norm_backward, dev, stream, dt, dt if rt is None else rt, op, ldo, yp, ldy, alpha, wt, wp, gt,
             gp, gr, gc, np_, ldn, hp, ldh, w2p, dyp, lddy, rp, ldr, dwp, dgt, dgp, dgr, dgc, dw2, T, cols, eps,
             eps if next_eps is None else next_eps, sp, sn)
