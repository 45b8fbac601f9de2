"""What a network is trained with, on torch tensors: ``layer_norm``,
``dropout``, ``linear_cross_entropy`` and their gradients.

Marshalling only, by the rules of ``feed_forward.py``: the HIP kernels of
``libmiconv.so`` on torch's current stream of the tensors' device, outputs and
workspaces as torch allocations on that stream, rows at any pitch and
alignment, contiguous arguments that fit each other through ``_native.so``.
"""
import collections
import operator

import torch

import convolution_forward_conv2d_amd as mic
from . import feed_forward as ff
from .feed_forward import (E4M3, _CODE, _call, _empty, _even, _flag, _gpu, _handle, _matrix, _ptr, _rows, _vector, _weights,
                           _workspace)

LayerNorm = collections.namedtuple("LayerNorm", ["y", "sum", "mean", "rstd", "scale"])
LayerNorm.__doc__ = """layer_norm's results: y; sum = x + residual (x itself without a residual), mean and rstd, fp32 per
row, which layer_norm_backward takes; scale, fp32 per row, where y is e4m3 (else None)."""

LinearCrossEntropy = collections.namedtuple("LinearCrossEntropy", ["loss", "lse", "count"])
LinearCrossEntropy.__doc__ = """linear_cross_entropy's results: loss, fp32; lse, the logarithm of each row's sum of
exponentials, fp32 per row, and count, the number of rows that have a target (None without a reduction), which
linear_cross_entropy_backward takes."""

_FLOATS = (torch.float32, torch.bfloat16)


def _native():
    return ff._native or ff._load()


def _per_row(t, rows, device, what):
    if t.dtype != torch.float32 or t.device != device or t.numel() != rows or not t.is_contiguous():
        raise ValueError("%s must be %d packed fp32 values on %s" % (what, rows, device))
    return t.data_ptr()


def _whole(v, name):
    if isinstance(v, (bool, torch.Tensor)) or not hasattr(v, "__index__"):
        raise TypeError("%s must be a whole number, got %s" % (name, type(v).__name__))
    return operator.index(v)


# ---------------------------------------------------------------- norm

def layer_norm(x, weight, bias=None, residual=None, eps=1e-5, out_dtype=None):
    """s = x + residual, y = (s - mean(s)) / sqrt(mean((s - mean(s))^2) + eps) * weight + bias over the last dimension.

    x, residual, weight, bias: fp32 or bf16, one type.  y has x's type, or is
    torch.float8_e4m3fn with a scale per row (y * scale is the value).
    Returns LayerNorm(y, sum, mean, rstd, scale).
    """
    e4m3 = out_dtype is E4M3
    if e4m3 or out_dtype is None or out_dtype is x.dtype:
        r = _native().layer_norm(x, weight, bias, residual, eps, e4m3)
        if r is not None:
            return LayerNorm(*r)
    _gpu(x, "x", _FLOATS)
    dtype, device = x.dtype, x.device
    out_dtype = dtype if out_dtype is None else out_dtype
    if out_dtype not in (dtype, E4M3):
        raise TypeError("out_dtype must be %s or %s, got %s" % (dtype, E4M3, out_dtype))
    cols = x.shape[-1] if x.dim() else 0
    if cols < 1:
        raise ValueError("x must have at least one feature")
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    rows, ldx = _rows(x, cols, "x")
    wp = _vector(weight, cols, dtype, device, "weight")
    bp = 0 if bias is None else _vector(bias, cols, dtype, device, "bias")
    ldr, total = 0, x
    h = _handle(device)
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("residual has shape %s, x %s" % (tuple(residual.shape), tuple(x.shape)))
        ldr = _matrix(residual, rows, cols, dtype, device, "residual")
        total = _empty(x.shape, x, dtype)
    y = _empty(x.shape, x, out_dtype)
    mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
    rstd = torch.empty_like(mean)
    scale = torch.empty_like(mean) if out_dtype is E4M3 else None
    _call("mic_layer_norm", h, _CODE[dtype], _CODE[out_dtype], rows, cols, eps, x.data_ptr(), ldx, _ptr(residual), ldr,
          wp, bp, y.data_ptr(), cols, 0 if residual is None else total.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(),
          _ptr(scale))
    return LayerNorm(y, total, mean, rstd, scale)


def layer_norm_backward(dy, sum, weight, mean, rstd, dsum=None, bias=False, need_dweight=True):
    """(dx, dweight, dbias) of layer_norm, from its sum, mean and rstd; dx is residual's gradient too.

    dsum: the gradient that reaches sum past the norm (added to dx).
    dbias is None unless bias is true, and dweight is where need_dweight is
    false: what is None is not computed.
    """
    r = _native().layer_norm_backward(dy, sum, weight, mean, rstd, dsum, bias, need_dweight)
    if r is not None:
        return r
    bias, need_dweight = _flag(bias, "bias"), _flag(need_dweight, "need_dweight")
    _gpu(dy, "dy", _FLOATS)
    dtype, device = dy.dtype, dy.device
    cols = dy.shape[-1] if dy.dim() else 0
    if cols < 1:
        raise ValueError("dy must have at least one feature")
    rows, lddy = _rows(dy, cols, "dy")
    lds = _matrix(sum, rows, cols, dtype, device, "sum")
    wp = _vector(weight, cols, dtype, device, "weight")
    mp, rp = _per_row(mean, rows, device, "mean"), _per_row(rstd, rows, device, "rstd")
    ldd = 0 if dsum is None else _matrix(dsum, rows, cols, dtype, device, "dsum")
    h = _handle(device)
    dx = _empty(dy.shape, dy, dtype)
    dweight = torch.empty_like(weight) if need_dweight else None
    dbias = torch.empty_like(weight) if bias else None
    ws, wsp, wsn = None, 0, 0
    if need_dweight or bias:
        ws, wsp, wsn = _workspace("mic_layer_norm_backward_workspace", h, dy, rows, cols)
    _call("mic_layer_norm_backward", h, _CODE[dtype], rows, cols, dy.data_ptr(), lddy, sum.data_ptr(), lds, wp, mp, rp,
          _ptr(dsum), ldd, dx.data_ptr(), cols, _ptr(dweight), _ptr(dbias), wsp, wsn)
    return dx, dweight, dbias


# ---------------------------------------------------------------- dropout

def _drop(x, p, seed, offset, residual, what):
    r = _native().dropout(x, p, seed, offset, residual)
    if r is not None:
        return r
    _gpu(x, what, _FLOATS)
    if isinstance(p, torch.Tensor) or not 0 <= p <= 1:
        raise ValueError("p must be a number from 0 to 1, got %s" % (p,))
    dtype, device = x.dtype, x.device
    state = 0
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.device != device or seed.shape != (2,) or not seed.is_contiguous():
            raise ValueError("seed must be a number, or two packed int64 values on %s" % device)
        state, seed = seed.data_ptr(), 0
    seed, offset = _whole(seed, "seed"), _whole(offset, "offset")
    for name, v in (("seed", seed), ("offset", offset)):
        if not 0 <= v < 1 << 64:
            raise ValueError("%s must be from 0 to 2^64 - 1, got %d" % (name, v))
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("residual has shape %s, %s %s" % (tuple(residual.shape), what, tuple(x.shape)))
    if x.is_contiguous() and (residual is None or residual.is_contiguous()):
        rows, cols = 1, x.numel()
        ldx = ldr = cols
        if residual is not None:
            if residual.dtype is not dtype:
                raise TypeError("residual must be %s, got %s" % (dtype, residual.dtype))
            if residual.device != device:
                raise ValueError("residual is on %s, not on %s" % (residual.device, device))
    else:
        cols = x.shape[-1]
        rows, ldx = _rows(x, cols, what)
        ldr = 0 if residual is None else _matrix(residual, rows, cols, dtype, device, "residual")
    h = _handle(device)
    y = _empty(x.shape, x, dtype)
    _call("mic_dropout", h, _CODE[dtype], rows, cols, float(p), seed, offset, state, x.data_ptr(), ldx, _ptr(residual), ldr,
          y.data_ptr(), cols)
    return y


def dropout(x, p, seed, offset=0, residual=None):
    """x / (1 - p) where an element is kept, 0 where it is dropped, + residual.

    An element is dropped with probability p, rounded to a multiple of 2^-16
    (and x scaled by what that makes of 1 / (1 - p)).  Which ones goes by
    seed, offset and the element's position in row-major order alone, so no
    mask is stored and dropout_backward takes the same three: a seed for the
    run, an offset for the layer and step.  seed may be an int64 tensor of two
    on x's device, the seed and what is added to offset: a captured call draws
    anew when that tensor has changed between replays.

    x, residual: fp32 or bf16, one type and shape.  residual's gradient is dy.
    """
    return _drop(x, p, seed, offset, residual, "x")


def dropout_backward(dy, p, seed, offset=0):
    """dx of dropout with the same p, seed and offset."""
    return _drop(dy, p, seed, offset, None, "dy")


# ---------------------------------------------------------------- loss

def _targets(target, shape, device):
    if target.dtype is not torch.int64:
        raise TypeError("target must be %s, got %s" % (torch.int64, target.dtype))
    if target.device != device:
        raise ValueError("target is on %s, not on %s" % (target.device, device))
    if target.shape != shape:
        raise ValueError("target has shape %s, expected %s" % (tuple(target.shape), tuple(shape)))
    if not target.is_contiguous():
        raise ValueError("target must be contiguous")
    return target.data_ptr()


def _loss_gradient(dloss, shape, rows, device):
    """Pointer to dloss, and whether it has a value for each row."""
    each = dloss.shape == shape and dloss.dim() > 0
    if each and not dloss.is_contiguous() and not any(st for n, st in zip(dloss.shape, dloss.stride()) if n > 1):
        dloss, each = dloss[(0,) * dloss.dim()], False         # one value, expanded: a sum's gradient
    return _per_row(dloss, rows if each else 1, device, "dloss"), each


def _smoothing(label_smoothing):
    if isinstance(label_smoothing, torch.Tensor) or not 0 <= label_smoothing < 1:
        raise ValueError("label_smoothing must be a number from 0 and below 1, got %s" % (label_smoothing,))
    return float(label_smoothing)


def _ignored(ignore_index):
    ignore_index = _whole(ignore_index, "ignore_index")
    if not -1 << 63 <= ignore_index < 1 << 63:
        raise ValueError("ignore_index does not fit int64")
    return ignore_index


def linear_cross_entropy(x, w, target, bias=None, reduction="mean", ignore_index=-100, label_smoothing=0.0):
    """The cross entropy of softmax(x w^T + bias) and one class per row, without keeping the logits.

    x (..., k), w (classes, k), bias (classes): fp32 or bf16, one type; target
    (...): int64.  With z the logits, a = label_smoothing:
        loss = log sum e^z - (1 - a) z[target] - a mean(z)
    per row (reduction "none"), its "sum" or its "mean" over the rows whose
    target is not ignore_index (0 over no rows).  A target that is neither
    that nor a class makes its loss NaN.
    Returns LinearCrossEntropy(loss, lse, count).
    """
    mode = mic.REDUCTIONS.get(reduction)
    if mode is not None:
        r = _native().linear_cross_entropy(x, w, target, bias, mode, ignore_index, label_smoothing)
        if r is not None:
            return LinearCrossEntropy(*r)
    _gpu(x, "x", _FLOATS)
    if mode is None:
        raise ValueError("unknown reduction %r (one of %s)" % (reduction, ", ".join(mic.REDUCTIONS)))
    dtype, device = x.dtype, x.device
    k = x.shape[-1] if x.dim() else 0
    m, ldx = _rows(x, k, "x")
    ldw = _weights(w, k, dtype, device, "w")
    n = w.shape[0]
    if n < 1:
        raise ValueError("w must have at least one class")
    bp = 0 if bias is None else _vector(bias, n, dtype, device, "bias")
    tp = _targets(target, x.shape[:-1], device)
    smoothing, ignore_index = _smoothing(label_smoothing), _ignored(ignore_index)
    h = _handle(device)
    lse = x.new_empty(x.shape[:-1], dtype=torch.float32)
    loss = torch.empty_like(lse) if mode == 0 else x.new_empty((), dtype=torch.float32)
    count = None if mode == 0 else torch.empty_like(loss)
    fn = "mic_linear_cross_entropy_workspace" + ("_aligned" if _even((x, ldx), (w, ldw)) else "")
    wk, wkp, wkn = _workspace(fn, h, x, _CODE[dtype], m, n, k)
    _call("mic_linear_cross_entropy", h, _CODE[dtype], mode, m, n, k, x.data_ptr(), ldx, w.data_ptr(), ldw, bp, tp,
          ignore_index, smoothing, loss.data_ptr(), lse.data_ptr(), _ptr(count), wkp, wkn)
    return LinearCrossEntropy(loss, lse, count)


def linear_cross_entropy_backward(dloss, x, w, target, lse, bias=None, count=None, ignore_index=-100, label_smoothing=0.0,
                                  need_dx=True, need_dw=True, need_dbias=True):
    """(dx, dw, dbias) of linear_cross_entropy, from its inputs and its lse and, of a mean, its count.

    dloss: the gradient of the loss, fp32, a single value or (reduction
    "none") one per row, packed or a single one expanded.  dbias is None without a bias; dx, dw and dbias are
    where need_dx, need_dw and need_dbias are false: what is None is not
    computed.  A row without a target has dx = 0 and adds 0 times its x to dw,
    which is no number where x is infinite or none: pad with finite rows.
    """
    r = _native().linear_cross_entropy_backward(dloss, x, w, target, lse, bias, count, ignore_index, label_smoothing,
                                                need_dx, need_dw, need_dbias)
    if r is not None:
        return r
    need_dx, need_dw, need_dbias = _flag(need_dx, "need_dx"), _flag(need_dw, "need_dw"), _flag(need_dbias, "need_dbias")
    _gpu(x, "x", _FLOATS)
    dtype, device = x.dtype, x.device
    k = x.shape[-1] if x.dim() else 0
    m, ldx = _rows(x, k, "x")
    ldw = _weights(w, k, dtype, device, "w")
    n = w.shape[0]
    if n < 1:
        raise ValueError("w must have at least one class")
    bp = 0 if bias is None else _vector(bias, n, dtype, device, "bias")
    tp, lp = _targets(target, x.shape[:-1], device), _per_row(lse, m, device, "lse")
    dp, each = _loss_gradient(dloss, x.shape[:-1], m, device)
    cp = 0 if count is None else _per_row(count, 1, device, "count")
    smoothing, ignore_index = _smoothing(label_smoothing), _ignored(ignore_index)
    h = _handle(device)
    dx = _empty(x.shape, x, dtype) if need_dx else None
    dw = _empty(w.shape, w, dtype) if need_dw else None
    dbias = torch.empty_like(bias) if need_dbias and bias is not None else None
    fn = "mic_linear_cross_entropy_backward_workspace" + ("_aligned" if _even((x, ldx), (w, ldw)) else "")
    wk, wkp, wkn = _workspace(fn, h, x, _CODE[dtype], m, n, k)
    _call("mic_linear_cross_entropy_backward", h, _CODE[dtype], m, n, k, dp, each, x.data_ptr(), ldx, w.data_ptr(), ldw, bp, tp,
          ignore_index, smoothing, lp, cp, _ptr(dx), k, _ptr(dw), k, _ptr(dbias), wkp, wkn)
    return dx, dw, dbias
