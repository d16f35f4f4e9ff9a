"""Checks and launch plumbing shared by the operator modules: a wrong type,
shape, stride or device is an error here, before any kernel.

A single-token call's kernels take a few microseconds, so the checks read
each tensor property once and compare plain integers."""
from __future__ import annotations

import torch

from . import binding as B

TYPES = {torch.bfloat16: B.MOE_T_BF16, torch.float16: B.MOE_T_F16, torch.float32: B.MOE_T_F32}
F32_ONLY = {torch.float32: B.MOE_T_F32}
BYTES = {B.MOE_T_BF16: 2, B.MOE_T_F16: 2, B.MOE_T_F32: 4}

_I32 = torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_grad_enabled = torch.is_grad_enabled


def _no_graph(name):
    raise ValueError(f"{name}: requires grad, and the call records no graph: call it under torch.no_grad(), or in the "
                     "forward and backward of a torch.autograd.Function")


def rows(name, t, dev, n, cols, types=TYPES):
    """A tensor of n rows (any number if None) of cols contiguous values on
    device index dev: (type code, address, row stride, address of its end)."""
    code = types.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: type {t.dtype} is not one of {[str(x) for x in types]}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (n is not None and shape[0] != n):
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [{'rows' if n is None else n}, {cols}]")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected device {dev}")
    if t.requires_grad and _grad_enabled():
        _no_graph(name)
    p, m = t.data_ptr(), shape[0]
    if m == 0:
        return code, p, cols, p
    step, one = t.stride()
    if m == 1:
        step = cols
    if (one != 1 and cols > 1) or step < cols:
        raise ValueError(f"{name}: rows have to be contiguous and must not overlap (strides {tuple(t.stride())})")
    return code, p, step, p + ((m - 1) * step + cols) * BYTES[code]


def whole(name, t, dev, dtype, shape=None):
    """Address of a contiguous tensor of one type and shape (None: the caller
    has looked at its shape)."""
    if t.dtype != dtype or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected {dtype} {tuple(shape or t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected device {dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: has to be contiguous")
    if dtype is not _I32 and t.requires_grad and _grad_enabled():
        _no_graph(name)
    return t.data_ptr()


def workspace(ws, need, x, stream):
    """Address and size of ws, or of one of need bytes on x's device, of the
    stream that will use it."""
    if ws is None and need and x.get_device() >= 0:
        if stream is None:
            ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        else:
            with torch.cuda.stream(stream):
                ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    return (None, 0) if ws is None else (whole("ws", ws, x.get_device(), torch.uint8), ws.numel())


def overlaps(name):
    raise ValueError(f"{name}: overlaps an input")


def launch(fn, dev, stream, *args):
    """fn(*args, stream) with the tensors' device current; stream: a torch
    stream of that device, or None for its current one."""
    if dev < 0:
        raise ValueError("tensors have to be on the GPU")
    if stream is None:
        s = _raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream of {stream.device}, tensors on device {dev}")
    else:
        s = stream.cuda_stream
    if dev == _current_device():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc < 0:
        B.check(rc)
