"""Sublayers in 8 bits: RMS norm with the residual and the cast, the casts, products,
the experts' layer for a few tokens.

The same kind of binding as the sublayer operators'.  8-bit tensors are E4M3
codes (uint8) with a scale for each block of 128 values of a row, or of 128 x 128
of a weight matrix: UE8M0 bytes (uint8), as the casts write them, or fp32.

The calls are short on the GPU, so their tensors are looked at by the module
_tensors (csrc/py_tensors.cpp), one call each; where something does not fit, the
checks below say what.
"""
from __future__ import annotations

import torch

from . import _lib
from .sublayer import (_DTYPE, _HALF, _NAMES, _at, _current_device, _dense, _like, _norm_input, _norm_weights, _out_rows,
                       _raw_stream, _rows, _scratch, _tensor)

__all__ = ["hc_fp8_cast", "hc_fp8_cast_weights", "hc_rms_norm", "hc_rms_norm_backward", "hc_fp8_mm",
           "hc_moe_tokens"]

RMS_NORM_EPS = 1e-6
FP8_BLOCK = 128  # values that share a scale

_SCALE = {torch.float32: 0, torch.uint8: 3}  # hc_dtype of scales
_SCALES = tuple(_SCALE)
_F32, _U8, _I32 = 0, 3, 4                    # types by the numbers of _tensors (fp32, bf16, fp16: hc_dtype's)
_SCALE_BITS = 1 << _F32 | 1 << _U8


def _changed():
    raise ValueError("a tensor does not fit the others")


def _blocks(d):
    return -(-d // FP8_BLOCK)


def _input(x, name):
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if x.dtype not in _DTYPE:
        raise TypeError("%s must be %s, got %s" % (name, _NAMES, x.dtype))


def _code_rows(codes, scales, shape, dev):
    """Given codes (evenly spaced rows) and scales of a shape; returns the codes' row stride."""
    _tensor(codes, "codes", (torch.uint8,), dev)
    if codes.shape != shape:
        raise ValueError("codes has shape %s, expected %s" % (tuple(codes.shape), tuple(shape)))
    _dense(scales, "scales", (torch.uint8,), (*shape[:-1], _blocks(shape[-1])), dev)
    return _rows(codes, "codes")[1]


def _pair(codes, scales):
    if (codes is None) != (scales is None):
        raise ValueError("codes and scales go together")


def hc_fp8_cast(x, codes=None, scales=None, stream=None):
    """Rows x [..., d] (fp32, bf16 or fp16; evenly spaced) -> (codes [..., d], scales
    [..., ceil(d / 128)]) uint8: E4M3 numbers with a power-of-two scale for every 128
    values of a row."""
    T = _lib.tensors()
    look = T.rows(x)
    if look is None or look[1] > 2:
        _input(x, "x")
        if x.dim() < 1 or x.shape[-1] < 1:
            raise ValueError("x must be [..., d] with d >= 1")
        _rows(x, "x")
        _tensor(x, "x")
        _changed()
    p, kind, dev, n, xs, d = look
    _pair(codes, scales)
    cs = d if codes is None else _code_rows(codes, scales, x.shape, x.device)
    if stream is not None or _current_device() != dev:
        with _at(x.device, stream):
            return hc_fp8_cast(x, codes, scales)
    if codes is None:
        lead = x.shape[:-1]
        codes, scales = T.empty(_U8, dev, *lead, d), T.empty(_U8, dev, *lead, -(-d // FP8_BLOCK))
    _lib.call("hc_fp8_cast", p, xs, kind, n, d, codes.data_ptr(), cs, scales.data_ptr(), _raw_stream(dev))
    return codes, scales


def hc_fp8_cast_weights(w, codes=None, scales=None, stream=None):
    """Weight matrices w [..., N, K] (fp32, bf16 or fp16, contiguous) -> (codes [..., N, K],
    scales [..., ceil(N / 128), ceil(K / 128)]) uint8: E4M3 numbers with a power-of-two
    scale for every block of 128 x 128."""
    _input(w, "w")
    if w.dim() < 2 or w.shape[-1] < 1 or w.shape[-2] < 1:
        raise ValueError("w must be [..., N, K] with N, K >= 1")
    _dense(w, "w", (w.dtype,), w.shape, w.device)
    dev, lead = w.device, w.shape[:-2]
    N, K = w.shape[-2:]
    s_shape = (*lead, _blocks(N), _blocks(K))
    _pair(codes, scales)
    if codes is not None:
        _dense(codes, "codes", (torch.uint8,), w.shape, dev)
        _dense(scales, "scales", (torch.uint8,), s_shape, dev)
    if stream is not None or _current_device() != dev.index:
        with _at(dev, stream):
            return hc_fp8_cast_weights(w, codes, scales)
    if codes is None:
        codes = torch.empty(w.shape, dtype=torch.uint8, device=dev)
        scales = torch.empty(s_shape, dtype=torch.uint8, device=dev)
    _lib.call("hc_fp8_cast_weights", w.data_ptr(), _DTYPE[w.dtype], lead.numel(), N, K, codes.data_ptr(), scales.data_ptr(),
              _raw_stream(dev.index))
    return codes, scales


def hc_rms_norm(x, norm_w, residual=None, norm_eps=RMS_NORM_EPS, out="y", r=None, y=None, codes=None, scales=None,
                return_rstd=False, stream=None):
    """RMS norm of x [..., d] (fp32, bf16 or fp16; evenly spaced rows), to which residual
    (of x's shape and type) is added first, with norm_w [d] (fp32 or x's type) -> a dict of
    y [..., d] of x's type (out "y" or "both"), codes and scales as hc_fp8_cast's of the
    unrounded y (out "fp8" or "both"), with a residual r = x + residual of x's type (the
    residual of the next norm and what the backward reads), with return_rstd rstd [...]
    fp32.  r, y, codes and scales may be given; r may be x or residual itself."""
    T = _lib.tensors()
    look = T.rows(x)
    w = None if look is None else T.dense(norm_w, 1 << look[1] | 1 << _F32, look[2], look[5])
    if w is None or look[1] > 2:
        _norm_weights(norm_w, None, x, _norm_input(x)[2])
        _changed()
    p, kind, dev, n, xs, d = look
    if out not in ("y", "fp8", "both"):
        raise ValueError('out must be "y", "fp8" or "both", got %r' % (out,))
    wide, narrow = out != "fp8", out != "y"
    q = None
    res_s = rs = ys = cs = d
    if residual is not None:
        more = T.rows(residual) if isinstance(residual, torch.Tensor) and residual.shape == x.shape else None
        if more is None or more[1] != kind or more[2] != dev:
            _like(residual, "residual", x, (x.dtype,))
            _changed()
        q, res_s = more[0], more[4]
    elif r is not None:
        raise ValueError("r is the sum with a residual: none is given")
    if (y is not None and not wide) or (codes is not None and not narrow):
        raise ValueError("out=%r does not write what is given" % out)
    _pair(codes, scales)
    if r is not None:
        rs = _like(r, "r", x, (x.dtype,))
    if y is not None:
        ys = _like(y, "y", x, (x.dtype,))
    if codes is not None:
        cs = _code_rows(codes, scales, x.shape, x.device)
    if stream is not None or _current_device() != dev:
        with _at(x.device, stream):
            return hc_rms_norm(x, norm_w, residual, norm_eps, out, r, y, codes, scales, return_rstd)
    shape, res = x.shape, {}
    lead = shape[:-1]
    if residual is not None:
        res["r"] = r = T.empty(kind, dev, *shape) if r is None else r
    if wide:
        res["y"] = y = T.empty(kind, dev, *shape) if y is None else y
    if narrow:
        if codes is None:
            codes, scales = T.empty(_U8, dev, *shape), T.empty(_U8, dev, *lead, -(-d // FP8_BLOCK))
        res["codes"], res["scales"] = codes, scales
    if return_rstd:
        res["rstd"] = T.empty(_F32, dev, *lead)
    _lib.call("hc_rms_norm", p, xs, q, res_s, kind, w, _DTYPE[norm_w.dtype], n, d, norm_eps, None if r is None else r.data_ptr(), rs,
              y.data_ptr() if wide else None, ys, codes.data_ptr() if narrow else None, cs,
              scales.data_ptr() if narrow else None, res["rstd"].data_ptr() if return_rstd else None, _raw_stream(dev))
    return res


def hc_rms_norm_backward(g_y, r, norm_w, rstd, g_r=None, g_x=None, workspace=None, stream=None):
    """The backward of hc_rms_norm: g_y [..., d] (fp32 or r's type), r (without a residual:
    x), norm_w, the forward's rstd, and g_r (of g_y's shape and type), the gradient that
    reaches r past the norm -> dict of g_x [..., d] of g_y's type, the gradient of x and of
    the residual, and g_norm_w [d] fp32, the sum over all rows.  A cast's gradient is that
    of the value it rounds.  g_x may be g_r itself.  workspace: a uint8 device tensor of at
    least the size the library asks for (allocated here when None)."""
    T = _lib.tensors()
    look, g = T.rows(r), T.rows(g_y)
    w = st = None
    if look is not None and g is not None:
        w = T.dense(norm_w, 1 << look[1] | 1 << _F32, look[2], look[5])
        st = T.dense(rstd, 1 << _F32, look[2], *r.shape[:-1])
    if w is None or st is None or look[1] > 2 or g[1] not in (_F32, look[1]) or g[2] != look[2] or g_y.shape != r.shape:
        d = _norm_input(r)[2]
        _norm_weights(norm_w, None, r, d)
        _like(g_y, "g_y", r, (torch.float32, r.dtype))
        _dense(rstd, "rstd", (torch.float32,), r.shape[:-1], r.device)
        _changed()
    p, kind, dev, n, rs, d = look
    grs = d if g_r is None else _like(g_r, "g_r", r, (g_y.dtype,))
    gxs = d if g_x is None else _like(g_x, "g_x", r, (g_y.dtype,))
    if workspace is not None:
        _scratch(workspace, r.device)
    if stream is not None or _current_device() != dev:
        with _at(r.device, stream):
            return hc_rms_norm_backward(g_y, r, norm_w, rstd, g_r, g_x, workspace)
    if g_x is None:
        g_x = T.empty(g[1], dev, *r.shape)
    if workspace is None:
        workspace = T.empty(_U8, dev, max(_lib.load().hc_rms_norm_backward_workspace_bytes(n, d), 16))
    g_w = T.empty(_F32, dev, d)
    _lib.call("hc_rms_norm_backward", g[0], g[4], None if g_r is None else g_r.data_ptr(), grs, g[1], p, rs, kind, w,
              _DTYPE[norm_w.dtype], st, n, d, g_x.data_ptr(), gxs, g_w.data_ptr(), workspace.data_ptr(), workspace.numel(),
              _raw_stream(dev))
    return {"g_x": g_x, "g_norm_w": g_w}


def hc_fp8_mm(x, x_scales, w, w_scales, transposed=False, y=None, out_dtype=None, workspace=None, stream=None):
    """Products of 8-bit numbers: x [M, K] codes (evenly spaced rows) with x_scales
    [M, ceil(K / 128)], w [N, K] codes with w_scales [ceil(N / 128), ceil(K / 128)]
    (scales UE8M0 bytes or fp32) -> y [M, N] of out_dtype (fp32, bf16, the default, or
    fp16), y = x w^T.  transposed: x [M, N] with x_scales [M, ceil(N / 128)] -> y [M, K] =
    x w, the gradient of the rows from the output's, cast by hc_fp8_cast (the weights' is
    hc_grouped_mm_weights of the 16-bit rows, as one expert's).  N and K are multiples of
    16.  workspace: a uint8 device tensor of at least the size the library asks for
    (allocated here when None)."""
    T = _lib.tensors()
    look = T.rows(x)
    sx = pw = sw = None
    if look is not None and isinstance(w, torch.Tensor) and w.dim() == 2 and x.dim() == 2:
        N, K = w.shape
        C, L = (K, N) if transposed else (N, K)
        dev, M = look[2], x.shape[0]
        pw = T.dense(w, 1 << _U8, dev, N, K)
        sx = T.dense(x_scales, _SCALE_BITS, dev, M, -(-L // FP8_BLOCK))
        sw = T.dense(w_scales, _SCALE_BITS, dev, -(-N // FP8_BLOCK), -(-K // FP8_BLOCK))
    if sx is None or pw is None or sw is None or look[1] != _U8 or look[5] != L:
        _mm_checks(x, x_scales, w, w_scales, transposed)
        _changed()
    p, _, dev, n, xs, _ = look
    xs = xs if n > 1 else max(16, -(-L // 16) * 16)  # (a single row may carry any stride)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if y is None else y.dtype
    if out_dtype not in _DTYPE:
        raise TypeError("out_dtype must be %s, got %s" % (_NAMES, out_dtype))
    kind = _DTYPE[out_dtype]
    ys = C if y is None else _out_rows(y, "y", (M, C), (out_dtype,), x.device)
    if workspace is not None:
        _scratch(workspace, x.device)
    if stream is not None or _current_device() != dev:
        with _at(x.device, stream):
            return hc_fp8_mm(x, x_scales, w, w_scales, transposed, y, out_dtype, workspace)
    if y is None:
        y = T.empty(kind, dev, M, C)
    if workspace is None:
        need = _lib.load().hc_fp8_mm_workspace_bytes(transposed, M, N, K)
        workspace = T.empty(_U8, dev, need) if need else None
    _lib.call("hc_fp8_mm", p, xs, sx, _SCALE[x_scales.dtype], pw, sw, _SCALE[w_scales.dtype], transposed, M, N, K, y.data_ptr(), ys,
              kind, None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
              _raw_stream(dev))
    return y


def _mm_checks(x, x_scales, w, w_scales, transposed):
    _tensor(x, "x", (torch.uint8,))
    dev = x.device
    _tensor(w, "w", (torch.uint8,), dev)
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [M, width] and w [N, K]")
    _dense(w, "w", (torch.uint8,), w.shape, dev)
    (N, K), M = w.shape, x.shape[0]
    L = N if transposed else K
    if x.shape[1] != L:
        raise ValueError("x has shape %s, expected (M, %d)" % (tuple(x.shape), L))
    _rows(x, "x")
    _dense(x_scales, "x_scales", _SCALES, (M, _blocks(L)), dev)
    _dense(w_scales, "w_scales", _SCALES, (_blocks(N), _blocks(K)), dev)


_SCORES = {"softmax": 0, "sigmoid": 1}


def hc_moe_tokens(x, w_up, w_down, ids=None, weights=None, logits=None, top_k=None, score="softmax", normalise=True,
                  scale=1.0, up_scales=None, down_scales=None, y=None, workspace=None, stream=None):
    """A whole mixture-of-experts layer for up to 64 tokens: x [T, d] (bf16 or fp16, evenly
    spaced rows), w_up [experts, 2, inner, d] (the gate's rows, then the other's) and w_down
    [experts, d, inner], of x's type, or uint8 codes with up_scales [experts, 2,
    ceil(inner / 128), ceil(d / 128)] and down_scales [experts, ceil(d / 128),
    ceil(inner / 128)] (UE8M0 bytes or fp32; hc_fp8_cast_weights makes both).  y[t] is the sum
    over t's experts of weight * w_down[e] (silu(w_up[e, 0] x[t]) * (w_up[e, 1] x[t])).

    The choice is given, ids [T, top_k] int32 and weights [T, top_k] fp32 (an id out of
    range, such as -1, counts for nothing): -> y [T, d].  Or it is made of logits
    [T, experts] fp32: the top_k largest, weighted by the softmax over all experts or
    the sigmoid (score), with normalise divided by their sum over the chosen ones,
    times scale: -> (y, ids, weights).  d and inner are multiples of 16.  For training and for
    more tokens: hc_grouped_mm.  workspace: a uint8 device tensor of at least the
    size the library asks for (allocated here when None)."""
    X = _lib.tensors()
    look = X.rows(x)
    fits = False
    if look is not None and look[1] in (1, 2) and x.dim() == 2 and isinstance(w_up, torch.Tensor) and w_up.dim() == 4:
        p, kind, dev, n, xs, d = look
        T, E, inner = x.shape[0], w_up.shape[0], w_up.shape[2]
        f8 = up_scales is not None
        bits = 1 << (_U8 if f8 else kind)
        up, down = X.dense(w_up, bits, dev, E, 2, inner, d), X.dense(w_down, bits, dev, E, d, inner)
        fits = up is not None and down is not None and (down_scales is not None) == f8
        us = ds = None
        if f8 and fits:
            bits = 1 << (_F32 if getattr(up_scales, "dtype", None) is torch.float32 else _U8)
            bi, bd = -(-inner // FP8_BLOCK), -(-d // FP8_BLOCK)
            us, ds = X.dense(up_scales, bits, dev, E, 2, bi, bd), X.dense(down_scales, bits, dev, E, bd, bi)
            fits = us is not None and ds is not None
        if fits and logits is not None:
            lg = X.dense(logits, 1 << _F32, dev, T, E)
            fits = lg is not None and ids is None and weights is None and score in _SCORES and isinstance(top_k, int) and top_k > 0
        elif fits:
            lg, fits = None, isinstance(ids, torch.Tensor) and ids.dim() == 2 and top_k in (None, ids.shape[1])
            if fits:
                top_k = ids.shape[1]
                fits = X.dense(ids, 1 << _I32, dev, T, top_k) is not None and X.dense(weights, 1 << _F32, dev, T, top_k) is not None
    if not fits:
        _moe_checks(x, w_up, w_down, ids, weights, logits, top_k, score, up_scales, down_scales)
        _changed()
    xs = xs if n > 1 else -(-d // 8) * 8  # (a single row may carry any stride)
    ys = d if y is None else _out_rows(y, "y", (T, d), (x.dtype,), x.device)
    if workspace is not None:
        _scratch(workspace, x.device)
    if stream is not None or _current_device() != dev:
        with _at(x.device, stream):
            return hc_moe_tokens(x, w_up, w_down, ids, weights, logits, None if logits is None else top_k, score, normalise,
                                 scale, up_scales, down_scales, y, workspace)
    if y is None:
        y = X.empty(kind, dev, T, d)
    if workspace is None:
        workspace = X.empty(_U8, dev, max(_lib.load().hc_moe_tokens_workspace_bytes(T, top_k, inner), 16))
    if logits is not None:
        ids, weights = X.empty(_I32, dev, T, top_k), X.empty(_F32, dev, T, top_k)
    _lib.call("hc_moe_tokens", p, xs, kind, T, d, E, inner, top_k, lg, _SCORES.get(score, 0), normalise, scale, ids.data_ptr(),
              weights.data_ptr(), up, down, 4 if f8 else kind, us, ds, _SCALE[up_scales.dtype] if f8 else 0, y.data_ptr(), ys,
              workspace.data_ptr(), workspace.numel(), _raw_stream(dev))
    return y if logits is None else (y, ids, weights)


def _moe_checks(x, w_up, w_down, ids, weights, logits, top_k, score, up_scales, down_scales):
    _tensor(x, "x", _HALF)
    dev = x.device
    if x.dim() != 2:
        raise ValueError("x must be [T, d]")
    T, d = x.shape
    _rows(x, "x")
    if (up_scales is None) != (down_scales is None):
        raise ValueError("up_scales and down_scales go together")
    f8 = up_scales is not None
    kinds = (torch.uint8,) if f8 else (x.dtype,)
    _tensor(w_up, "w_up", kinds, dev)
    if w_up.dim() != 4 or w_up.shape[1] != 2 or w_up.shape[3] != d:
        raise ValueError("w_up has shape %s, expected (experts, 2, inner, %d)" % (tuple(w_up.shape), d))
    E, inner = w_up.shape[0], w_up.shape[2]
    _dense(w_up, "w_up", kinds, w_up.shape, dev)
    _dense(w_down, "w_down", kinds, (E, d, inner), dev)
    if f8:
        _dense(up_scales, "up_scales", _SCALES, (E, 2, _blocks(inner), _blocks(d)), dev)
        _dense(down_scales, "down_scales", (up_scales.dtype,), (E, _blocks(d), _blocks(inner)), dev)
    if (logits is None) == (ids is None):
        raise ValueError("either logits or ids and weights")
    if logits is not None:
        if weights is not None:
            raise ValueError("weights are given with ids")
        if score not in _SCORES:
            raise ValueError('score must be "softmax" or "sigmoid", got %r' % (score,))
        if not isinstance(top_k, int) or top_k < 1:
            raise ValueError("top_k must be a number from 1 on")
        _dense(logits, "logits", (torch.float32,), (T, E), dev)
    else:
        _tensor(ids, "ids", (torch.int32,), dev)
        if ids.dim() != 2 or (top_k is not None and ids.shape[1] != top_k):
            raise ValueError("ids must be [T, top_k]")
        top_k = ids.shape[1]
        _dense(ids, "ids", (torch.int32,), (T, top_k), dev)
        _dense(weights, "weights", (torch.float32,), (T, top_k), dev)
