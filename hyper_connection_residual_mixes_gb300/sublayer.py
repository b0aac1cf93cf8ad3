"""Sublayer operators: layer norm, the experts' matrix products, AdamW.

The same kind of binding as the rest of the package: each function has the
name of the C entry point it calls (include/hc.h), checks and marshals
tensors, allocates outputs with PyTorch when they are not supplied and
enqueues the call on the current CUDA stream of the tensors' device, or on
``stream``.  What a call allocates belongs to the stream it runs on.
"""
from __future__ import annotations

import torch

from . import _lib

__all__ = ["hc_layer_norm", "hc_layer_norm_backward", "hc_grouped_mm", "hc_grouped_mm_weights",
           "hc_grouped_mm_backward", "adamw_state", "adamw_plan", "hc_adamw_step"]

LAYER_NORM_EPS = 1e-5

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_NAMES = "torch.float32, torch.bfloat16 or torch.float16"


def _tensor(t, name, dtypes=None, device=None):
    if t.__class__ is not torch.Tensor and not isinstance(t, torch.Tensor):
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
    if t.shape != shape:
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
    if len(shape) == 2 and strides[1] == 1 and shape[0] > 1:
        return shape[0], strides[0]
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


# the stream a device's current work goes to, as the number the C ABI takes
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch.cuda.current_device


def _at(device, stream):
    """The context in which a call for `device` runs on `stream` (None: the
    device's current stream); what is allocated inside belongs to that stream."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError("stream is on %s, the tensors are on %s" % (stream.device, device))
    return torch.cuda.stream(stream)


def _norm_weights(norm_w, norm_b, x, d):
    _dense(norm_w, "norm_w", (torch.float32, x.dtype), (d,), x.device)
    if norm_b is not None:
        _dense(norm_b, "norm_b", (norm_w.dtype,), (d,), x.device)


def _norm_input(x):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dtype not in _DTYPE:
        raise TypeError("x must be %s, got %s" % (_NAMES, x.dtype))
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., d] with d >= 1")
    n, step = _rows(x, "x")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor (libhc has no CPU path)")
    return n, step, x.shape[-1]


def _like(t, name, x, dtypes):
    """Rows of x's shape; returns their stride."""
    _tensor(t, name, dtypes, x.device)
    if t.shape != x.shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(x.shape)))
    return _rows(t, name)[1]


def hc_layer_norm(x, norm_w, norm_b=None, norm_eps=LAYER_NORM_EPS, y=None, return_stats=False, stream=None):
    """Layer norm of x [..., d] (fp32, bf16 or fp16; evenly spaced rows) with
    norm_w, norm_b [d] (fp32 or x's type; norm_b optional) -> y [..., d] of x's
    type [+ (mean, rstd) [...] fp32 for the backward when return_stats]."""
    n, xs, d = _norm_input(x)
    _norm_weights(norm_w, norm_b, x, d)
    dev = x.device
    ys = d if y is None else _like(y, "y", x, (x.dtype,))
    if stream is not None or _current_device() != dev.index:
        with _at(dev, stream):
            return hc_layer_norm(x, norm_w, norm_b, norm_eps, y, return_stats)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    mean = rstd = None
    if return_stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    _lib.call("hc_layer_norm", x.data_ptr(), xs, _DTYPE[x.dtype], norm_w.data_ptr(),
              None if norm_b is None else norm_b.data_ptr(), _DTYPE[norm_w.dtype], n, d, norm_eps, y.data_ptr(), ys,
              None if mean is None else mean.data_ptr(), None if rstd is None else rstd.data_ptr(),
              _raw_stream(dev.index))
    return (y, mean, rstd) if return_stats else y


def hc_layer_norm_backward(g_y, x, norm_w, mean, rstd, bias=True, g_x=None, workspace=None, stream=None):
    """The backward of hc_layer_norm: g_y [..., d] (fp32 or x's type), x, norm_w and
    the forward's mean, rstd -> dict of g_x [..., d] of g_y's type and the sums
    over all rows g_norm_w [d] and (unless bias is False) g_norm_b [d], fp32.
    Of a norm on the path's h (h_pre_out) g_x is the gradient of h = sum_s pre_mix[s]
    x[s], which hc_block_step_backward does not take: add pre_mix[s] g_x to its
    g_x[s] and <g_x, x[s]> to its g_pre_mix[s].
    workspace: a uint8 device tensor of at least the size the library asks for
    (allocated here when None)."""
    n, xs, d = _norm_input(x)
    dev = x.device
    _norm_weights(norm_w, None, x, d)
    gs = _like(g_y, "g_y", x, (torch.float32, x.dtype))
    _dense(mean, "mean", (torch.float32,), x.shape[:-1], dev)
    _dense(rstd, "rstd", (torch.float32,), x.shape[:-1], dev)
    gxs = d if g_x is None else _like(g_x, "g_x", x, (g_y.dtype,))
    if workspace is not None:
        _scratch(workspace, dev)
    if stream is not None or _current_device() != dev.index:
        with _at(dev, stream):
            return hc_layer_norm_backward(g_y, x, norm_w, mean, rstd, bias, g_x, workspace)
    if g_x is None:
        g_x = torch.empty(x.shape, dtype=g_y.dtype, device=dev)
    if workspace is None:
        need = _lib.load().hc_layer_norm_backward_workspace_bytes(n, d)
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    g_w = torch.empty((d,), dtype=torch.float32, device=dev)
    g_b = torch.empty((d,), dtype=torch.float32, device=dev) if bias else None
    _lib.call("hc_layer_norm_backward", g_y.data_ptr(), gs, _DTYPE[g_y.dtype], x.data_ptr(), xs, _DTYPE[x.dtype],
              norm_w.data_ptr(), _DTYPE[norm_w.dtype], mean.data_ptr(), rstd.data_ptr(), n, d, g_x.data_ptr(), gxs,
              g_w.data_ptr(), None if g_b is None else g_b.data_ptr(), workspace.data_ptr(), workspace.numel(),
              _raw_stream(dev.index))
    return {"g_x": g_x, "g_norm_w": g_w, "g_norm_b": g_b} if bias else {"g_x": g_x, "g_norm_w": g_w}


def _scratch(workspace, dev):
    _tensor(workspace, "workspace", (torch.uint8,), dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


_HALF = (torch.bfloat16, torch.float16)


def _grouped(rows, name, w_shape, offsets):
    """The checks shared by the grouped products: rows [n, width] of 16-bit values,
    the weights' shape, offsets.  Returns (n, row stride)."""
    if not isinstance(rows, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if rows.dtype not in _HALF:
        raise TypeError("%s must be torch.bfloat16 or torch.float16, got %s" % (name, rows.dtype))
    if rows.dim() != 2 or len(w_shape) != 3:
        raise ValueError("%s must be [n, width] and the weights [experts, ., .]" % name)
    n, step = _rows(rows, name)
    if not rows.is_cuda:
        raise ValueError("%s must be a CUDA tensor (libhc has no CPU path)" % name)
    _dense(offsets, "offsets", (torch.int32,), (w_shape[0] + 1,), rows.device)
    # (a single row may carry any stride)
    return n, step if n > 1 else rows.shape[1]


def _out_rows(y, name, shape, types, dev):
    _tensor(y, name, types, dev)
    if tuple(y.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(y.shape), tuple(shape)))
    n, step = _rows(y, name)
    return step if n > 1 else shape[-1]


def hc_grouped_mm(x, w, offsets, transposed=False, y=None, out_dtype=None, workspace=None, stream=None):
    """Products of rows grouped by expert: x [n, K] (bf16 or fp16, rows sorted by
    expert), w [experts, N, K] of x's type (with transposed [experts, K, N]),
    offsets [experts + 1] int32 on the device -> y [n, N] of out_dtype (x's type
    or fp32), y[r] = w[e] x[r] for offsets[e] <= r < offsets[e + 1].  Rows of no
    expert are zeros in a y made here and stay as they are in a y given.
    workspace: a uint8 device tensor of at least the size the library asks for
    (allocated here when None)."""
    _tensor(w, "w")
    n, xs = _grouped(x, "x", w.shape, offsets)
    dev = x.device
    E, K = w.shape[0], x.shape[1]
    N = w.shape[2] if transposed else w.shape[1]
    _dense(w, "w", (x.dtype,), (E, K, N) if transposed else (E, N, K), dev)
    if out_dtype is None:
        out_dtype = x.dtype if y is None else y.dtype
    if out_dtype is not x.dtype and out_dtype is not torch.float32:
        raise TypeError("out_dtype must be %s or torch.float32, got %s" % (x.dtype, out_dtype))
    ys = N if y is None else _out_rows(y, "y", (n, N), (out_dtype,), dev)
    if workspace is not None:
        _scratch(workspace, dev)
    if stream is not None or _current_device() != dev.index:
        with _at(dev, stream):
            return hc_grouped_mm(x, w, offsets, transposed, y, out_dtype, workspace)
    zero = y is None
    if zero:
        y = torch.empty((n, N), dtype=out_dtype, device=dev)
    if workspace is None:
        need = _lib.load().hc_grouped_mm_workspace_bytes(n, E, N, K)
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    _lib.call("hc_grouped_mm", x.data_ptr(), xs, w.data_ptr(), transposed, offsets.data_ptr(), n, E, N, K,
              _DTYPE[x.dtype], y.data_ptr(), ys, _DTYPE[out_dtype], zero,
              None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
              _raw_stream(dev.index))
    return y


def hc_grouped_mm_weights(g_y, x, offsets, transposed=False, g_w=None, out_dtype=None, workspace=None, stream=None):
    """The weights' gradient of hc_grouped_mm: g_y [n, N] and x [n, K] of one type ->
    g_w [experts, N, K] (transposed: [experts, K, N]) of out_dtype (x's type or
    fp32), the sum over each expert's rows of g_y[r] x[r]^T.  workspace: a uint8
    device tensor of at least the size the library asks for (allocated here when
    None)."""
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be [experts + 1]")
    E = offsets.shape[0] - 1
    n, xs = _grouped(x, "x", (E, 0, 0), offsets)
    dev = x.device
    _tensor(g_y, "g_y", (x.dtype,), dev)
    if g_y.dim() != 2 or g_y.shape[0] != n:
        raise ValueError("g_y has shape %s, expected (%d, N)" % (tuple(g_y.shape), n))
    gs = _rows(g_y, "g_y")[1] if n > 1 else g_y.shape[1]
    N, K = g_y.shape[1], x.shape[1]
    shape = (E, K, N) if transposed else (E, N, K)
    if out_dtype is None:
        out_dtype = x.dtype if g_w is None else g_w.dtype
    if out_dtype is not x.dtype and out_dtype is not torch.float32:
        raise TypeError("out_dtype must be %s or torch.float32, got %s" % (x.dtype, out_dtype))
    if g_w is not None:
        _dense(g_w, "g_w", (out_dtype,), shape, dev)
    if workspace is not None:
        _scratch(workspace, dev)
    if stream is not None or _current_device() != dev.index:
        with _at(dev, stream):
            return hc_grouped_mm_weights(g_y, x, offsets, transposed, g_w, out_dtype, workspace)
    if g_w is None:
        g_w = torch.empty(shape, dtype=out_dtype, device=dev)
    if workspace is None:
        need = _lib.load().hc_grouped_mm_weights_workspace_bytes(n, E, N, K)
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    _lib.call("hc_grouped_mm_weights", g_y.data_ptr(), gs, x.data_ptr(), xs, offsets.data_ptr(), n, E, N, K,
              _DTYPE[x.dtype], g_w.data_ptr(), transposed, _DTYPE[out_dtype],
              None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
              _raw_stream(dev.index))
    return g_w


def hc_grouped_mm_backward(g_y, x, w, offsets, transposed=False, g_x=None, g_w=None, stream=None):
    """Both gradients of hc_grouped_mm(x, w, offsets, transposed): a dict of g_x
    [n, K] (rows of no expert as hc_grouped_mm's) and g_w of w's shape."""
    return {"g_x": hc_grouped_mm(g_y, w, offsets, not transposed, y=g_x, stream=stream),
            "g_w": hc_grouped_mm_weights(g_y, x, offsets, transposed, g_w=g_w, stream=stream)}


STATE_GROUP = 32  # values of a tensor that share a scale in the 8-bit states


def adamw_state(p, mxfp8=False):
    """Zero states (m, v) for a parameter: fp32 tensors of its shape, or with mxfp8
    pairs (codes uint8 of its shape, scales uint8 [ceil(numel / 32)])."""
    if not mxfp8:
        return (torch.zeros(p.shape, dtype=torch.float32, device=p.device),
                torch.zeros(p.shape, dtype=torch.float32, device=p.device))
    groups = -(-p.numel() // STATE_GROUP)
    return tuple((torch.zeros(p.shape, dtype=torch.uint8, device=p.device),
                  torch.zeros((groups,), dtype=torch.uint8, device=p.device)) for _ in range(2))


class AdamwPlan:
    """The tensors of hc_adamw_step, checked and described once (adamw_plan).  It
    keeps them alive; a tensor whose storage has moved since (t.data = ...) is
    described anew by the next step, one of another shape, type or order is
    refused, also where it begins at the same place."""

    def __init__(self, fields, device):
        self._fields = fields      # (tensor, index of the description, its member, shape, dtype)
        self._tensors = [f[0] for f in fields]
        self.device = device
        self.count = 1 + max((f[1] for f in fields), default=-1)
        self._array = (_lib.AdamwTensor * self.count)()
        self._at = None
        self._snapshot = _lib.snapshot()

    def _describe(self):
        # (every step looks at sizes, strides and types too: a pointer alone does not tell a tensor
        # from its first values, its transpose or another type's view of it)
        at = self._snapshot(self._tensors)
        if at == self._at:
            return
        # (all of them before the first is described: a refusal leaves the old descriptions whole)
        for t, i, member, shape, dtype in self._fields:
            if t.shape != shape or t.dtype != dtype or t.device != self.device or not t.is_contiguous():
                raise ValueError("%s of tensor %d has changed since the plan was made" % (member, i))
        for t, i, member, shape, dtype in self._fields:
            setattr(self._array[i], member, t.data_ptr())
            if member == "p":
                self._array[i].numel = shape.numel()
            if member in ("p", "g", "p_copy"):
                setattr(self._array[i], "copy_type" if member == "p_copy" else member + "_type", _DTYPE[dtype])
        self._at = at


def adamw_plan(params, grads, exp_avg, exp_avg_sq, copies=None):
    """The plan of hc_adamw_step: lists of equal length of contiguous CUDA tensors
    on one device.  params[i] fp32, bf16 or fp16; grads[i] of its shape, fp32 or
    its type; exp_avg[i], exp_avg_sq[i] as adamw_state makes them (fp32, or
    (codes, scales) pairs); copies[i] (optional, None where there is none): a
    bf16 or fp16 tensor that receives an fp32 parameter's new value rounded.
    The step reads the gradients where these tensors are: a gradient that a
    call has allocated anew is copied into its tensor (or that call given the
    tensor to write to) before the step."""
    params, grads, exp_avg, exp_avg_sq = list(params), list(grads), list(exp_avg), list(exp_avg_sq)
    copies = [None] * len(params) if copies is None else list(copies)
    if not params:
        raise ValueError("params is empty")
    if not len(params) == len(grads) == len(exp_avg) == len(exp_avg_sq) == len(copies):
        raise ValueError("params, grads, exp_avg, exp_avg_sq and copies must have one entry per parameter")
    for i, (p, g, m, v, c) in enumerate(zip(params, grads, exp_avg, exp_avg_sq, copies)):
        for t, name in ((p, "params"), (g, "grads")):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s[%d] must be a torch.Tensor" % (name, i))
        if p.dtype not in _DTYPE:
            raise TypeError("params[%d] must be %s, got %s" % (i, _NAMES, p.dtype))
        if isinstance(m, torch.Tensor) != isinstance(v, torch.Tensor):
            raise TypeError("exp_avg[%d] and exp_avg_sq[%d] must be of one kind" % (i, i))
        if c is not None and p.dtype != torch.float32:
            raise TypeError("copies[%d]: only fp32 parameters have one" % i)
    dev = params[0].device if isinstance(params[0], torch.Tensor) else None
    fields = []
    for i, (p, g, m, v, c) in enumerate(zip(params, grads, exp_avg, exp_avg_sq, copies)):
        def field(t, name, member, dtypes, shape):
            _dense(t, "%s[%d]" % (name, i), dtypes, shape, dev)
            fields.append((t, i, member, t.shape, t.dtype))
        field(p, "params", "p", (p.dtype,), p.shape)
        field(g, "grads", "g", (torch.float32, p.dtype) if p.dtype != torch.float32 else (torch.float32,), p.shape)
        for s, name, member in ((m, "exp_avg", "m"), (v, "exp_avg_sq", "v")):
            if isinstance(s, torch.Tensor):
                field(s, name, member, (torch.float32,), p.shape)
            else:
                field(s[0], name, member, (torch.uint8,), p.shape)
                field(s[1], name + " scales", member + "_scales", (torch.uint8,), (-(-p.numel() // STATE_GROUP),))
        if c is not None:
            field(c, "copies", "p_copy", (torch.bfloat16, torch.float16), p.shape)
    return AdamwPlan(fields, dev)


def hc_adamw_step(plan, lr, step, betas=(0.9, 0.999), adam_eps=1e-8, weight_decay=0.01, grad_scale=None, stream=None):
    """One AdamW step over the plan's tensors, in place.  lr is a number or a
    one-element fp32 CUDA tensor, step a number from 1 on or a one-element int64
    CUDA tensor (so that a captured step reads the current ones); grad_scale, a
    one-element fp32 CUDA tensor, multiplies the gradients."""
    if not isinstance(plan, AdamwPlan):
        raise TypeError("plan must come from adamw_plan")
    dev = plan.device
    on_device = []
    for t, name, dtype in ((lr, "lr", torch.float32), (step, "step", torch.int64), (grad_scale, "grad_scale", torch.float32)):
        if t.__class__ is not float and t.__class__ is not int and isinstance(t, torch.Tensor):
            _tensor(t, name, (dtype,), dev)
            if t.numel() != 1:
                raise ValueError("%s must have one element" % name)
            on_device.append(t.data_ptr())
        else:
            on_device.append(None)
    if grad_scale is not None and on_device[2] is None:
        raise TypeError("grad_scale must be a CUDA tensor")
    if stream is not None or _current_device() != dev.index:
        with _at(dev, stream):
            return hc_adamw_step(plan, lr, step, betas, adam_eps, weight_decay, grad_scale)
    plan._describe()
    _lib.call("hc_adamw_step", plan._array, plan.count, 0.0 if on_device[0] else lr, betas[0], betas[1], adam_eps,
              weight_decay, 1 if on_device[1] else step, on_device[0], on_device[1], on_device[2],
              _raw_stream(dev.index))
