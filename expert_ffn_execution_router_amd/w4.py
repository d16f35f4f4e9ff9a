"""Products of a few rows with 4-bit weights in groups of inputs sharing a
scale (and zero point): W[n, c] = (q[n, c] - zero[n, c / group]) * scale[n, c / group].

codes: uint8 [N, K/2] (or [E, N, K/2], one matrix per expert), two codes per
byte, even input in the low nibble.  scales: bf16 or fp16 [..., N, K/group];
zeros: the same shape in x's type, or None for 8.  group: 32, 64 or a
multiple of 128.  x: bf16 or fp16, out: x's type or fp32.  gated: the matrix
is [gate; up] stacked and out = silu(x gate^T) * (x up^T).  x is finite, in
bf16 below 2^116 with zeros of up to 16 (fp32 holds |x| (q + |zero|) summed
over 128 inputs; past it a row may be infinite or NaN where the result is not).

The memory from out's first to its last value must not meet an input's.  No
call records a graph: with gradients enabled, a tensor that requires grad is
refused.
moe_w4_matmul in include/moe.h has the details; calls enqueue on the current
stream of the tensors' device (or `stream`) and can be captured.
"""
from __future__ import annotations

import torch

from . import _args as A
from . import binding as B

_X = {torch.bfloat16: B.MOE_T_BF16, torch.float16: B.MOE_T_F16}
_I32 = torch.int32


def _matmul(x, dev, xshape, out, codes, scales, zeros, gated, E, row_map, map_div, offsets, counts, n, stream):
    K, lead, sshape = xshape[-1], codes.shape[:-1], scales.shape
    xt, xp, ldx, xe = A.rows("x", x, dev, None, K, _X)
    groups, st = sshape[-1], _X.get(scales.dtype)
    if sshape[:-1] != lead or groups < 1 or K % groups:
        raise ValueError(f"scales: shape {tuple(sshape)}, expected {tuple(lead)} + (K/group,) with K = {K}")
    if st is None:
        raise ValueError(f"scales: type {scales.dtype}, expected bf16 or fp16")
    N = lead[-1]
    cp = A.whole("codes", codes, dev, torch.uint8, (*lead, K // 2))
    sp = A.whole("scales", scales, dev, scales.dtype)
    zp = None if zeros is None else A.whole("zeros", zeros, dev, x.dtype, sshape)
    ot, op, ldo, oe = A.rows("out", out, dev, n, N // 2 if gated else N)
    if xp < oe and op < xe:
        A.overlaps("out")
    A.launch(B.lib().moe_w4_matmul, dev, stream, xt, xp, ldx, xshape[0], row_map, map_div, offsets, counts, E, n, cp,
             st, sp, zp, N, K, K // groups, 1 if gated else 0, ot, op, ldo)


def linear(x, out, codes, scales, zeros=None, gated=False, stream=None):
    """out = x W^T for x [T, K] and one matrix (codes [N, K/2])."""
    if codes.dim() != 2:
        raise ValueError(f"codes: shape {tuple(codes.shape)}, expected [N, K/2]")
    shape = x.shape
    _matmul(x, x.get_device(), shape, out, codes, scales, zeros, gated, 1, None, 1, None, None, shape[0], stream)


def experts(x, offsets, out, codes, scales, zeros=None, counts=None, row_map=None, map_div=1, gated=False,
            stream=None):
    """Grouped rows times their expert's matrix (codes [E, N, K/2]): rows
    offsets[e] .. + counts[e] of out (counts None: up to offsets[e + 1]) from
    the same rows of x, or with row_map from x rows row_map[r] // map_div.
    Rows in no segment stay as they were."""
    if codes.dim() != 3:
        raise ValueError(f"codes: shape {tuple(codes.shape)}, expected [E, N, K/2]")
    if map_div >> 31:
        raise ValueError(f"map_div: {map_div}, need 1 <= map_div < 2^31")
    dev, shape, E, n = x.get_device(), x.shape, codes.shape[0], out.shape[0]
    op = A.whole("offsets", offsets, dev, _I32, (E + 1,))
    cp = None if counts is None else A.whole("counts", counts, dev, _I32, (E,))
    mp = None if row_map is None else A.whole("row_map", row_map, dev, _I32, (n,))
    if row_map is None and shape[0] < n:
        raise ValueError(f"x: {shape[0]} rows, out has {n}")
    _matmul(x, dev, shape, out, codes, scales, zeros, gated, E, mp, map_div, op, cp, n, stream)
