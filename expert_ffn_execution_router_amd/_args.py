"""Checks and launch plumbing shared by the operator modules (dispatch, w4):
a wrong type, shape, stride or device is an error here, before any kernel."""
from __future__ import annotations

import torch

from . import binding as B

TYPES = {torch.bfloat16: B.MOE_T_BF16, torch.float16: B.MOE_T_F16, torch.float32: B.MOE_T_F32}


def rows(name, t, device, cols=None, types=TYPES):
    """A [n, cols] tensor with contiguous rows: (type code, row stride)."""
    if t.dtype not in types:
        raise ValueError(f"{name}: type {t.dtype} is not one of {[str(x) for x in types]}")
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [rows{'' if cols is None else f', {cols}'}]")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    n, c = t.shape
    step = t.stride(0) if n > 1 else c
    if n and ((c > 1 and t.stride(1) != 1) or step < c):
        raise ValueError(f"{name}: rows have to be contiguous and must not overlap (strides {tuple(t.stride())})")
    return types[t.dtype], step


def whole(name, t, device, dtype, shape):
    """A contiguous tensor of one type and shape."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected {dtype} {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: has to be contiguous")
    return t.data_ptr()


def apart(name, out, *others):
    """out must not share memory with what the kernels read while writing it."""
    a0 = out.data_ptr()
    a1 = a0 + _span(out)
    for t in others:
        if t is not None and t.data_ptr() < a1 and a0 < t.data_ptr() + _span(t):
            raise ValueError(f"{name}: overlaps an input")


def _span(t):
    if t.numel() == 0:
        return 0
    return (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def launch(fn, device, stream, *args):
    """fn(*args, stream) with device current; stream: a torch stream of that
    device, or None for its current one."""
    if device.type != "cuda":
        raise ValueError(f"tensors have to be on the GPU, got {device}")
    if stream is not None and stream.device != device:
        raise ValueError(f"stream of {stream.device}, tensors on {device}")
    s = torch.cuda.current_stream(device) if stream is None else stream
    if device.index == torch.cuda.current_device():
        return B.check(fn(*args, s.cuda_stream))
    with torch.cuda.device(device):
        return B.check(fn(*args, s.cuda_stream))
