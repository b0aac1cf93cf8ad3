"""Sublayer operators: layer norm, the experts' matrix products, AdamW.

The same kind of binding as the rest of the package: each function has the
name of the C entry point it calls (include/hc.h), checks and marshals
tensors, allocates outputs with PyTorch when they are not supplied and
enqueues the call on the current CUDA stream of the tensors' device, or on
``stream``.  What a call allocates belongs to the stream it runs on.
"""
from __future__ import annotations

import contextlib

import torch

from . import _lib

__all__ = ["hc_layer_norm", "hc_layer_norm_backward"]

LAYER_NORM_EPS = 1e-5

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_NAMES = "torch.float32, torch.bfloat16 or torch.float16"


def _tensor(t, name, dtypes=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (libhc has no CPU path)" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    return t


def _dense(t, name, dtypes, shape, device):
    """A contiguous tensor of a given shape."""
    _tensor(t, name, dtypes, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _rows(t, name):
    """(rows, row stride) of a tensor [..., d] whose last axis is dense and whose
    leading axes are evenly spaced rows (a slice of one stream, of a wider
    buffer, a broadcast row); anything else is refused."""
    shape, strides = t.shape, t.stride()
    d = shape[-1]
    if d > 1 and strides[-1] != 1:
        raise ValueError("%s must be dense along its last axis" % name)
    n, step = 1, None
    for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size == 1:
            continue
        if size == 0:
            return 0, d
        if step is None:
            step = stride
        elif stride != step * n:
            raise ValueError("%s must have evenly spaced rows" % name)
        n *= size
    return n, d if step is None else step


def _on(device, stream):
    """The device and stream a call runs on, as a context and the raw stream."""
    if stream is not None:
        if stream.device != device:
            raise ValueError("stream is on %s, the tensors are on %s" % (stream.device, device))
        return torch.cuda.stream(stream), stream.cuda_stream
    raw = torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.current_device() == device.index:
        return contextlib.nullcontext(), raw
    return torch.cuda.device(device), raw


def _norm_weights(norm_w, norm_b, x, d):
    types = (torch.float32, x.dtype) if x.dtype != torch.float32 else (torch.float32,)
    _dense(norm_w, "norm_w", types, (d,), x.device)
    if norm_b is not None:
        _dense(norm_b, "norm_b", (norm_w.dtype,), (d,), x.device)


def _norm_input(x):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dtype not in _DTYPE:
        raise TypeError("x must be %s, got %s" % (_NAMES, x.dtype))
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., d] with d >= 1")
    return x


def hc_layer_norm(x, norm_w, norm_b=None, norm_eps=LAYER_NORM_EPS, y=None, return_stats=False, stream=None):
    """Layer norm of x [..., d] (fp32, bf16 or fp16; evenly spaced rows) with
    norm_w, norm_b [d] (fp32 or x's type; norm_b optional) -> y [..., d] of x's
    type [+ (mean, rstd) [...] fp32 for the backward when return_stats]."""
    _norm_input(x)
    n, xs = _rows(x, "x")
    d = x.shape[-1]
    _tensor(x, "x")
    _norm_weights(norm_w, norm_b, x, d)
    dev = x.device
    if y is not None:
        _tensor(y, "y", (x.dtype,), dev)
        if y.shape != x.shape:
            raise ValueError("y has shape %s, expected %s" % (tuple(y.shape), tuple(x.shape)))
    ctx, raw = _on(dev, stream)
    with ctx:
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=dev)
            ys = d
        else:
            ys = _rows(y, "y")[1]
        mean = rstd = None
        if return_stats:
            mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
            rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        _lib.call("hc_layer_norm", x.data_ptr(), xs, _DTYPE[x.dtype], norm_w.data_ptr(),
                  None if norm_b is None else norm_b.data_ptr(), _DTYPE[norm_w.dtype], n, d, norm_eps,
                  y.data_ptr(), ys, None if mean is None else mean.data_ptr(),
                  None if rstd is None else rstd.data_ptr(), raw)
    return (y, mean, rstd) if return_stats else y


def hc_layer_norm_backward(g_y, x, norm_w, mean, rstd, bias=True, g_x=None, workspace=None, stream=None):
    """The backward of hc_layer_norm: g_y [..., d] (fp32 or x's type), x, norm_w and
    the forward's mean, rstd -> dict of g_x [..., d] of g_y's type and the sums
    over all rows g_norm_w [d] and (unless bias is False) g_norm_b [d], fp32."""
    _norm_input(x)
    n, xs = _rows(x, "x")
    d = x.shape[-1]
    _tensor(x, "x")
    dev = x.device
    _norm_weights(norm_w, None, x, d)
    _tensor(g_y, "g_y", (torch.float32, x.dtype), dev)
    if g_y.shape != x.shape:
        raise ValueError("g_y has shape %s, expected %s" % (tuple(g_y.shape), tuple(x.shape)))
    gs = _rows(g_y, "g_y")[1]
    _dense(mean, "mean", (torch.float32,), x.shape[:-1], dev)
    _dense(rstd, "rstd", (torch.float32,), x.shape[:-1], dev)
    if g_x is not None:
        _tensor(g_x, "g_x", (g_y.dtype,), dev)
        if g_x.shape != x.shape:
            raise ValueError("g_x has shape %s, expected %s" % (tuple(g_x.shape), tuple(x.shape)))
    if workspace is not None:
        _tensor(workspace, "workspace", (torch.uint8,), dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    need = _lib.load().hc_layer_norm_backward_workspace_bytes(n, d)
    ctx, raw = _on(dev, stream)
    with ctx:
        if g_x is None:
            g_x = torch.empty(x.shape, dtype=g_y.dtype, device=dev)
            gxs = d
        else:
            gxs = _rows(g_x, "g_x")[1]
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        sums = torch.empty((2 if bias else 1, d), dtype=torch.float32, device=dev)
        g_w, g_b = sums[0], sums[1] if bias else None
        _lib.call("hc_layer_norm_backward", g_y.data_ptr(), gs, _DTYPE[g_y.dtype], x.data_ptr(), xs,
                  _DTYPE[x.dtype], norm_w.data_ptr(), _DTYPE[norm_w.dtype], mean.data_ptr(), rstd.data_ptr(),
                  n, d, g_x.data_ptr(), gxs, g_w.data_ptr(), None if g_b is None else g_b.data_ptr(),
                  workspace.data_ptr(), workspace.numel(), raw)
    out = {"g_x": g_x, "g_norm_w": g_w}
    if bias:
        out["g_norm_b"] = g_b
    return out
