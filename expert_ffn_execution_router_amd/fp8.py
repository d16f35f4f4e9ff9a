"""Block-scaled 8-bit values on torch tensors: quantisation, products and
gradients, and a whole MoE layer for a few tokens.

Codes are torch.float8_e4m3fn with one fp32 scale per group of 128:

    rows        codes [rows, P(cols)], scales [P(cols)/128, rows]
    transposed  codes_t [cols, P(rows)], scales_t [P(rows)/128, cols]
    weights     codes [N, P(K)], scales [P(N)/128, P(K)/128] (or [E, ...]),
                transposed codes_t [K, P(N)], scales_t [P(K)/128, P(N)/128]

where P(n) = padded(n) is n rounded up to a multiple of 128; the padding is
zeros.  The caller owns every tensor; results go into tensors it passes.  Calls
enqueue on the current stream of the tensors' device (or `stream`, which the
caller orders after the work that made the inputs) and can be captured.  A
result's memory must not meet an input's or another result's.  No call records
a graph: with gradients enabled, a tensor that requires grad is refused.
include/moe.h has the details of each call under its C name.

Experts' forward and backward around dispatch.sort(..., align=128):

    quantize(x, xq, sx, xq_t, sx_t, row_map=perm, map_div=k)
    experts(xq, sx, offsets, *gate_up, z, counts=counts)
    quantize(z, aq, sa, aq_t, sa_t, row_map=perm, map_div=0, gated=True)
    experts(aq, sa, offsets, *down, y, counts=counts)

    quantize(dy, dq, sd, dq_t, sd_t)            # dy from unpermute_backward
    experts(dq, sd, offsets, *down_t, da, counts=counts)
    weight_gradient(dq_t, sd_t, aq_t, sa_t, ddown, offsets=offsets)
    gated_backward(z, da, dz)
    quantize(dz, zq, sz, zq_t, sz_t, row_map=perm, map_div=0)
    experts(zq, sz, offsets, *gate_up_t, dxs, counts=counts)
    weight_gradient(zq_t, sz_t, xq_t, sx_t, dgate_up, offsets=offsets)
"""
from __future__ import annotations

import torch

from . import _args as A
from . import binding as B

_I32, _F32, F8 = torch.int32, torch.float32, torch.float8_e4m3fn
_16 = {torch.bfloat16: B.MOE_T_BF16, torch.float16: B.MOE_T_F16}


def padded(n: int) -> int:
    """n rounded up to whole groups."""
    return (n + 127) // 128 * 128


def _pair(name, codes, scales, dev, cshape, sshape):
    """Addresses of codes and their scales."""
    if codes is None or scales is None:
        if codes is None and scales is None:
            return None, None
        raise ValueError(f"{name}: codes and scales come together")
    return A.whole(name, codes, dev, F8, cshape), A.whole(f"scales of {name}", scales, dev, _F32, sshape)


def quantize(x, codes=None, scales=None, codes_t=None, scales_t=None, row_map=None, map_div=1, gated=False,
             stream=None):
    """Codes and scales of the rows of x (bf16, fp16 or fp32), transposed ones,
    or both.  gated: of silu(x[:, :n]) * x[:, n:].  row_map (int32): row r is x
    row row_map[r] // map_div (map_div 0: row r), zeros where it is -1; rows
    with a smaller entry keep their codes and scales."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected rows")
    dev, (n, width) = x.get_device(), x.shape
    if gated and width % 2:
        raise ValueError(f"x: {width} columns, gated rows have an even number")
    if map_div >> 31:
        raise ValueError(f"map_div: {map_div}, need 0 <= map_div < 2^31")
    cols = width // 2 if gated else width
    rows = row_map.numel() if row_map is not None else n
    dt, xp, ldx, _ = A.rows("x", x, dev, None, width)
    cp, sp = _pair("codes", codes, scales, dev, (rows, padded(cols)), (padded(cols) // 128, rows))
    ct, st = _pair("codes_t", codes_t, scales_t, dev, (cols, padded(rows)), (padded(rows) // 128, cols))
    mp = None if row_map is None else A.whole("row_map", row_map, dev, _I32, (rows,))
    A.launch(B.lib().moe_fp8_quantize, dev, stream, dt, xp, ldx, n, mp, map_div, 1 if gated else 0, rows, cols, cp, sp,
             ct, st)


def quantize_weights(w, codes=None, scales=None, codes_t=None, scales_t=None, stream=None):
    """Codes and block scales of w [N, K] or [E, N, K] (contiguous), of its
    transposes, or both."""
    if w.dim() not in (2, 3):
        raise ValueError(f"w: shape {tuple(w.shape)}, expected [N, K] or [E, N, K]")
    dev, (N, K), lead = w.get_device(), w.shape[-2:], tuple(w.shape[:-2])
    dt = A.TYPES.get(w.dtype)
    if dt is None:
        raise ValueError(f"w: type {w.dtype} is not one of {[str(x) for x in A.TYPES]}")
    wp = A.whole("w", w, dev, w.dtype)
    Np, Kp = padded(N), padded(K)
    cp, sp = _pair("codes", codes, scales, dev, (*lead, N, Kp), (*lead, Np // 128, Kp // 128))
    ct, st = _pair("codes_t", codes_t, scales_t, dev, (*lead, K, Np), (*lead, Kp // 128, Np // 128))
    A.launch(B.lib().moe_fp8_quantize_weights, dev, stream, dt, wp, lead[0] if lead else 1, N, K, cp, sp, ct, st)


def gated_backward(z, da, dz, stream=None):
    """dz = gradient of silu(gate) * up at z = [gate, up] rows, given da."""
    if z.dim() != 2 or z.shape[1] % 2:
        raise ValueError(f"z: shape {tuple(z.shape)}, expected [rows, 2 I]")
    dev, (n, width) = z.get_device(), z.shape
    dt, zp, ldz, _ = A.rows("z", z, dev, n, width)
    at, ap, lda, _ = A.rows("da", da, dev, n, width // 2)
    ot, op, ldo, _ = A.rows("dz", dz, dev, n, width)
    if at != dt or ot != dt:
        raise ValueError(f"da, dz: types {da.dtype}, {dz.dtype}, z has {z.dtype}")
    A.launch(B.lib().moe_gated_backward, dev, stream, dt, zp, ldz, ap, lda, n, width // 2, op, ldo)


def _matmul(a, a_scales, offsets, w, w_scales, out, counts, E, stream):
    if a.dim() != 2:
        raise ValueError(f"a: shape {tuple(a.shape)}, expected [rows, K]")
    dev, (n, K), lead, N = a.get_device(), a.shape, tuple(w.shape[:-2]), w.shape[-2]
    if K % 128:
        raise ValueError(f"a: {K} columns, expected whole groups of 128")
    G = K // 128
    ap, asp = _pair("a", a, a_scales, dev, (n, K), (G, n))
    wp, wsp = _pair("w", w, w_scales, dev, (*lead, N, K), (*lead, padded(N) // 128, G))
    ot, op, ldo, _ = A.rows("out", out, dev, n, N)
    A.launch(B.lib().moe_fp8_matmul, dev, stream, ap, asp, offsets, counts, E, n, wp, wsp, N, K, ot, op, ldo)


def linear(a, a_scales, w, w_scales, out, stream=None):
    """out = a w^T: rows' codes [R, K], weights' codes [N, K], out [R, N] in
    bf16, fp16 or fp32."""
    if w.dim() != 2:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected [N, K]")
    _matmul(a, a_scales, None, w, w_scales, out, None, 1, stream)


def experts(a, a_scales, offsets, w, w_scales, out, counts=None, stream=None):
    """Grouped rows times their expert's matrix (w [E, N, K]): rows offsets[e]
    .. + counts[e] (counts None: up to offsets[e + 1]).  Rows in no segment stay
    as they were."""
    if w.dim() != 3:
        raise ValueError(f"w: shape {tuple(w.shape)}, expected [E, N, K]")
    dev, E = a.get_device(), w.shape[0]
    op = A.whole("offsets", offsets, dev, _I32, (E + 1,))
    cp = None if counts is None else A.whole("counts", counts, dev, _I32, (E,))
    _matmul(a, a_scales, op, w, w_scales, out, cp, E, stream)


def weight_gradient_workspace_bytes(E: int, rows: int, N: int, K: int) -> int:
    return B.moe_fp8_weight_gradient_workspace_bytes(E, rows, N, K)


def weight_gradient(dy_t, dy_scales, x_t, x_scales, dw, offsets=None, add=False, ws=None, stream=None):
    """dw = dy^T x (or dw + dy^T x) from the transposed codes of dy [N, P(R)]
    and x [K, P(R)]: fp32 [N, K], or [E, N, K] over the rows offsets[e] ..
    offsets[e + 1] (multiples of 128).  ws: uint8 tensor of
    weight_gradient_workspace_bytes for P(R) rows; None allocates one where it
    is needed."""
    if dy_t.dim() != 2 or x_t.dim() != 2 or dw.dim() != (2 if offsets is None else 3):
        raise ValueError(f"dw: shape {tuple(dw.shape)}, expected [N, K], or [E, N, K] with offsets")
    dev, (N, rows), K = dy_t.get_device(), dy_t.shape, x_t.shape[0]
    if rows % 128:
        raise ValueError(f"dy_t: {rows} rows, expected whole groups of 128")
    E = 1 if offsets is None else dw.shape[0]
    dp, dsp = _pair("dy_t", dy_t, dy_scales, dev, (N, rows), (rows // 128, N))
    xp, xsp = _pair("x_t", x_t, x_scales, dev, (K, rows), (rows // 128, K))
    shape = (N, K) if offsets is None else (E, N, K)
    wp = A.whole("dw", dw, dev, _F32, shape)
    op = None if offsets is None else A.whole("offsets", offsets, dev, _I32, (E + 1,))
    sp, sn = A.workspace(ws, B.moe_fp8_weight_gradient_workspace_bytes(E, rows, N, K), x_t, stream)
    A.launch(B.lib().moe_fp8_weight_gradient, dev, stream, dp, dsp, xp, xsp, op, E, rows, N, K, 1 if add else 0, wp, K,
             sp, sn)


def layer_workspace_bytes(T: int, E: int, k: int, H: int, I: int) -> int:
    return B.moe_fp8_layer_workspace_bytes(T, E, k, H, I)


def layer(x, router, gate_up, gate_up_scales, down, down_scales, out, ids, weights, bias=None, base=None, ws=None,
          stream=None):
    """A whole MoE layer for up to 16 tokens x [T, H] (bf16 or fp16): router
    fp32 [E, H], gate_up [E, 2 I, H] and down [E, H, I] codes with block scales;
    ids int32 and weights fp32 [T, k] receive the routing, out [T, H] (x's type
    or fp32) the sum over the choices, on top of base (fp32 [T, H]).  ws: uint8
    tensor of layer_workspace_bytes, one for each call that may run at the same
    time; None allocates one."""
    if x.dim() != 2 or router.dim() != 2 or gate_up.dim() != 3 or ids.dim() != 2:
        raise ValueError("expected x [T, H], router [E, H], gate_up [E, 2 I, H], ids [T, k]")
    dev, (T, H), E, k, I = x.get_device(), x.shape, router.shape[0], ids.shape[1], gate_up.shape[1] // 2
    if H % 128 or I % 128 or H < 1 or I < 1:
        raise ValueError(f"H = {H}, I = {I}: expected multiples of 128")
    xt, xp, ldx, _ = A.rows("x", x, dev, T, H, _16)
    rp = A.whole("router", router, dev, _F32, (E, H))
    bp = None if bias is None else A.whole("bias", bias, dev, _F32, (E,))
    gp, gs = _pair("gate_up", gate_up, gate_up_scales, dev, (E, 2 * I, H), (E, I // 64, H // 128))
    dp, ds = _pair("down", down, down_scales, dev, (E, H, I), (E, H // 128, I // 128))
    ot, op, ldo, _ = A.rows("out", out, dev, T, H)
    ap, ldb = None, 0
    if base is not None:
        _, ap, ldb, _ = A.rows("base", base, dev, T, H, A.F32_ONLY)
    ip, wp = A.whole("ids", ids, dev, _I32, (T, k)), A.whole("weights", weights, dev, _F32, (T, k))
    sp, sn = A.workspace(ws, 0 if ws is not None else B.moe_fp8_layer_workspace_bytes(T, E, k, H, I), x, stream)
    A.launch(B.lib().moe_fp8_layer, dev, stream, xt, xp, ldx, rp, bp, T, E, k, H, I, gp, gs, dp, ds, ap, ldb, ot, op,
             ldo, ip, wp, sp, sn)
