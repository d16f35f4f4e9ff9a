"""Products of a few rows with 4-bit weights in groups of inputs sharing a
scale (and zero point): W[n, c] = (q[n, c] - zero[n, c / group]) * scale[n, c / group].

codes: uint8 [N, K/2] (or [E, N, K/2], one matrix per expert), two codes per
byte, even input in the low nibble.  scales: bf16 or fp16 [..., N, K/group];
zeros: the same shape in x's type, or None for 8.  group: 32, 64 or a
multiple of 128.  x: bf16 or fp16, out: x's type or fp32.  gated: the matrix
is [gate; up] stacked and out = silu(x gate^T) * (x up^T).

moe_w4_matmul in include/moe.h has the details; calls enqueue on the current
stream of the tensors' device (or `stream`) and can be captured.
"""
from __future__ import annotations

import torch

from . import _args as A
from . import binding as B

_X = {torch.bfloat16: B.MOE_T_BF16, torch.float16: B.MOE_T_F16}


def _matmul(x, out, codes, scales, zeros, gated, E, row_map, map_div, offsets, counts, stream):
    dev = x.device
    xt, ldx = A.rows("x", x, dev, None, _X)
    K = x.shape[1]
    lead, N = codes.shape[:-1], codes.shape[-2]
    if scales.dim() != codes.dim() or scales.shape[:-1] != lead or scales.shape[-1] < 1 or K % scales.shape[-1]:
        raise ValueError(f"scales: shape {tuple(scales.shape)}, expected {tuple(lead)} + (K/group,) with K = {K}")
    if scales.dtype not in _X:
        raise ValueError(f"scales: type {scales.dtype}, expected bf16 or fp16")
    group = K // scales.shape[-1]
    cp = A.whole("codes", codes, dev, torch.uint8, lead + (K // 2,))
    sp = A.whole("scales", scales, dev, scales.dtype, scales.shape)
    zp = None if zeros is None else A.whole("zeros", zeros, dev, x.dtype, scales.shape)
    ot, ldo = A.rows("out", out, dev, N // 2 if gated else N)
    A.apart("out", out, x)
    A.launch(B.moe_w4_matmul, dev, stream, xt, x.data_ptr(), ldx, x.shape[0], row_map, map_div, offsets, counts, E,
             out.shape[0], cp, _X[scales.dtype], sp, zp, N, K, group, 1 if gated else 0, ot, out.data_ptr(), ldo)


def linear(x, out, codes, scales, zeros=None, gated=False, stream=None):
    """out = x W^T for x [T, K] and one matrix (codes [N, K/2])."""
    if codes.dim() != 2:
        raise ValueError(f"codes: shape {tuple(codes.shape)}, expected [N, K/2]")
    if out.shape[0] != x.shape[0]:
        raise ValueError(f"out: {out.shape[0]} rows, x has {x.shape[0]}")
    _matmul(x, out, codes, scales, zeros, gated, 1, None, 1, None, None, stream)


def experts(x, offsets, out, codes, scales, zeros=None, counts=None, row_map=None, map_div=1, gated=False,
            stream=None):
    """Grouped rows times their expert's matrix (codes [E, N, K/2]): rows
    offsets[e] .. + counts[e] of out (counts None: up to offsets[e + 1]) from
    the same rows of x, or with row_map from x rows row_map[r] // map_div.
    Rows in no segment stay as they were."""
    if codes.dim() != 3:
        raise ValueError(f"codes: shape {tuple(codes.shape)}, expected [E, N, K/2]")
    dev, E, rows = x.device, codes.shape[0], out.shape[0]
    op = A.whole("offsets", offsets, dev, torch.int32, (E + 1,))
    np_ = None if counts is None else A.whole("counts", counts, dev, torch.int32, (E,))
    mp = None if row_map is None else A.whole("row_map", row_map, dev, torch.int32, (rows,))
    if row_map is None and x.shape[0] < rows:
        raise ValueError(f"x: {x.shape[0]} rows, out has {rows}")
    _matmul(x, out, codes, scales, zeros, gated, E, mp, map_div, op, np_, stream)
