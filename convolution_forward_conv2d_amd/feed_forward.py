"""The feed-forward operators on torch tensors: ``rms_norm``, ``linear``,
``gated_linear`` and their gradients.

Argument marshalling only, as for the convolutions: every step runs in the
HIP kernels of ``libmiconv.so``, on torch's current stream of the tensors'
device.  Outputs and workspaces are torch allocations on that stream, so the
calls may be captured into graphs.  Contiguous arguments that fit each other
pass through ``_native.so`` (csrc/binding.cpp), which takes half of Python's
time over a small call; all others, and wrong ones, through the checks here.

Activations ``x`` have any leading dimensions before their features; weights
are ``(out_features, in_features)``.  Features must be consecutive in memory
(stride 1) and the leading dimensions must flatten to one row pitch; rows may
be any distance apart and aligned to their element only.
"""
import collections
import threading

import torch

import convolution_forward_conv2d_amd as mic

E4M3 = torch.float8_e4m3fn
_CODE = {torch.float32: 0, torch.bfloat16: 2, E4M3: 3}

RmsNorm = collections.namedtuple("RmsNorm", ["y", "sum", "rstd", "scale"])
RmsNorm.__doc__ = """rms_norm's results: y; sum = x + residual (x itself without a residual) and rstd, fp32 per row,
which rms_norm_backward takes; scale, fp32 per row, where y is e4m3 (else None)."""

_native = None
_local = threading.local()
_bytes_of = {}
_fns = {}


def _load():
    global _native
    mic.lib()                                  # says what to do where nothing is built
    from . import _native as module
    _native = module
    return module


def _handle(device):
    """This thread's library handle on `device`, bound to torch's current stream there."""
    dev = device.index
    if dev != torch._C._cuda_getDevice():
        raise ValueError("tensors are on %s, the current device is cuda:%d" % (device, torch.cuda.current_device()))
    handles = _local.__dict__
    h = handles.get(dev)
    if h is None:
        h = handles[dev] = [mic.mic_create(), None]
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if stream != h[1]:
        status = mic.lib().mic_set_stream(h[0], stream)
        if status:
            raise mic.MicError(status, "mic_set_stream")
        h[1] = stream
    return h[0]


def _empty(shape, like, dtype):
    """torch.empty on like's device; the calls below cost a third of its dispatch."""
    if like.shape == shape and like.is_contiguous():
        return torch.empty_like(like, dtype=dtype)
    return like.new_empty(shape, dtype=dtype)


def _rows(t, cols, what):
    """t as (rows of `cols`, row pitch in elements), or why it cannot be read as one matrix."""
    shape = t.shape
    if len(shape) == 2 and shape[1] == cols and t.is_contiguous():
        return shape[0], cols
    strides = t.stride()
    if not shape or shape[-1] != cols:
        raise ValueError("%s has shape %s, expected (..., %d)" % (what, tuple(shape), cols))
    if cols > 1 and strides[-1] != 1 and t.numel():
        raise ValueError("%s: features must be consecutive in memory (stride 1)" % what)
    if len(shape) == 2:
        rows, pitch = shape[0], strides[0] if shape[0] > 1 else cols
    else:
        rows, pitch, expect = 1, cols, None
        for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
            if size > 1:
                if expect is None:
                    pitch = stride
                elif stride != expect and t.numel():
                    raise ValueError("%s: its leading dimensions do not flatten to one row pitch" % what)
                expect = stride * size
            rows *= size
    if pitch < cols:
        if t.numel():
            raise ValueError("%s: rows overlap (pitch %d, %d features)" % (what, pitch, cols))
        pitch = cols
    return rows, pitch


def _matrix(t, rows, cols, dtype, device, what):
    """Pitch of t, checked to be rows x cols of dtype on device."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, not on %s" % (what, t.device, device))
    n, pitch = _rows(t, cols, what)
    if n != rows:
        raise ValueError("%s has %d rows, expected %d" % (what, n, rows))
    return pitch


def _vector(t, size, dtype, device, what):
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, not on %s" % (what, t.device, device))
    if t.shape != (size,) or not (t.is_contiguous() or size < 2):
        raise ValueError("%s must be a packed vector of %d, got %s" % (what, size, tuple(t.shape)))
    return t.data_ptr()


def _gpu(t, what, types):
    if t.dtype not in types:
        raise TypeError("unsupported %s dtype %s" % (what, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % what)


def _weights(w, k, dtype, device, what):
    if w.dim() != 2:
        raise ValueError("%s must be (out_features, in_features)" % what)
    return _matrix(w, w.shape[0], k, dtype, device, what)


def _even(*matrices):
    """Whether every (tensor, pitch) has rows that count as aligned, so a call on them copies none."""
    return all((t.data_ptr() | pitch * t.element_size()) % 16 == 0 and pitch * t.element_size() < 1 << 22
               for t, pitch in matrices)


def _workspace(fn, h, like, *sizes):
    key = (fn, like.device.index, sizes)
    n = _bytes_of.get(key)
    if n is None:
        if len(_bytes_of) > 4096:
            _bytes_of.clear()
        n = _bytes_of[key] = getattr(mic, fn)(h, *sizes)
    if n == 0:
        return None, 0, 0
    t = like.new_empty(n, dtype=torch.uint8)
    return t, t.data_ptr(), n


def _call(name, *args):
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(mic.lib(), name)
    status = fn(*args)
    if status:
        raise mic.MicError(status, name)


def _act(activation):
    try:
        return mic.ACTIVATIONS[activation]
    except KeyError:
        raise ValueError("unknown activation %r (one of %s)" % (activation, ", ".join(mic.ACTIVATIONS))) from None


def _flag(v, name):
    if isinstance(v, torch.Tensor) and (v.dtype is not torch.bool or v.numel() != 1):
        raise TypeError("%s must be True or False, not a tensor" % name)
    return bool(v)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


# ---------------------------------------------------------------- norm

def rms_norm(x, weight, residual=None, eps=1e-6, out_dtype=None):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the last dimension.

    x, residual, weight: fp32 or bf16, one type.  y has x's type, or is
    torch.float8_e4m3fn with a scale per row (y * scale is the value).
    Returns RmsNorm(y, sum, rstd, scale).
    """
    e4m3 = out_dtype is E4M3
    if e4m3 or out_dtype is None or out_dtype is x.dtype:
        r = (_native or _load()).rms_norm(x, weight, residual, eps, e4m3)
        if r is not None:
            return RmsNorm(*r)
    _gpu(x, "x", (torch.float32, torch.bfloat16))
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
    ldr, total = 0, x
    h = _handle(device)
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("residual has shape %s, x %s" % (tuple(residual.shape), tuple(x.shape)))
        ldr = _matrix(residual, rows, cols, dtype, device, "residual")
        total = _empty(x.shape, x, dtype)
    y = _empty(x.shape, x, out_dtype)
    rstd = x.new_empty(x.shape[:-1], dtype=torch.float32)
    scale = torch.empty_like(rstd) if out_dtype is E4M3 else None
    _call("mic_rms_norm", h, _CODE[dtype], _CODE[out_dtype], rows, cols, eps, x.data_ptr(), ldx, _ptr(residual), ldr,
          wp, y.data_ptr(), cols, 0 if residual is None else total.data_ptr(), cols, rstd.data_ptr(), _ptr(scale))
    return RmsNorm(y, total, rstd, scale)


def rms_norm_backward(dy, sum, weight, rstd, dsum=None, need_dweight=True):
    """(dx, dweight) of rms_norm, from its sum and rstd; dx is residual's gradient too.

    dsum: the gradient that reaches sum past the norm (added to dx).
    dweight is None, and not computed, where need_dweight is false.
    """
    r = (_native or _load()).rms_norm_backward(dy, sum, weight, rstd, dsum, need_dweight)
    if r is not None:
        return r
    need_dweight = _flag(need_dweight, "need_dweight")
    _gpu(dy, "dy", (torch.float32, torch.bfloat16))
    dtype, device = dy.dtype, dy.device
    cols = dy.shape[-1] if dy.dim() else 0
    if cols < 1:
        raise ValueError("dy must have at least one feature")
    rows, lddy = _rows(dy, cols, "dy")
    lds = _matrix(sum, rows, cols, dtype, device, "sum")
    wp = _vector(weight, cols, dtype, device, "weight")
    if rstd.dtype != torch.float32 or rstd.device != device or rstd.numel() != rows or not rstd.is_contiguous():
        raise ValueError("rstd must be %d packed fp32 values on %s" % (rows, device))
    ldd = 0 if dsum is None else _matrix(dsum, rows, cols, dtype, device, "dsum")
    h = _handle(device)
    dx = _empty(dy.shape, dy, dtype)
    dweight = torch.empty_like(weight) if need_dweight else None
    ws, wsp, wsn = _workspace("mic_rms_norm_backward_workspace", h, dy, rows, cols) if need_dweight else (None, 0, 0)
    _call("mic_rms_norm_backward", h, _CODE[dtype], rows, cols, dy.data_ptr(), lddy, sum.data_ptr(), lds, wp,
          rstd.data_ptr(), _ptr(dsum), ldd, dx.data_ptr(), cols, _ptr(dweight), wsp, wsn)
    return dx, dweight


# ---------------------------------------------------------------- layers

def _wide(x, out_dtype):
    """Whether an e4m3 layer's outputs are fp32; None where out_dtype does not go with x."""
    if out_dtype is None or out_dtype is x.dtype:
        return None if out_dtype is E4M3 else False
    if x.dtype is E4M3 and out_dtype in (torch.bfloat16, torch.float32):
        return out_dtype is torch.float32
    return None


def _layer_types(x, out_dtype, scales):
    """The output type of a layer on x, with its scales checked to be there or not."""
    _gpu(x, "x", tuple(_CODE))
    if x.dtype is E4M3:
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("out_dtype must be bfloat16 or float32 for e4m3 operands, got %s" % out_dtype)
        if any(s is None for s in scales):
            raise ValueError("e4m3 operands need their scales, x's per row and the weights' per output feature")
        return out_dtype
    if out_dtype not in (None, x.dtype):
        raise TypeError("out_dtype must be x's, %s, got %s" % (x.dtype, out_dtype))
    if any(s is not None for s in scales):
        raise ValueError("scales are for e4m3 operands")
    return x.dtype


def _row_scale(x_scale, rows, device):
    if x_scale is None:
        return 0
    if (x_scale.dtype != torch.float32 or x_scale.device != device or x_scale.numel() != rows
            or not x_scale.is_contiguous()):
        raise ValueError("x_scale must be %d packed fp32 values on %s" % (rows, device))
    return x_scale.data_ptr()


def linear(x, w, bias=None, residual=None, activation="none", x_scale=None, w_scale=None, out_dtype=None,
           return_preact=False, fast_sums=False):
    """y = activation(x w^T + bias) + residual.

    x (..., k), w (n, k): fp32 or bf16, or both e4m3 with x_scale (per row)
    and w_scale (per output feature).  bias (n) and residual (..., n) have
    the output's type (out_dtype: for e4m3 operands bf16, the default, or
    fp32).  return_preact: (y, z) with z = x w^T + bias, for linear_backward.
    fast_sums: let the e4m3 matrix instruction add the products, at up to
    twice the rate but in sums shorter than fp32 (off by up to 2^-11 of the
    largest of 64 products); only e4m3 operands have that choice.
    """
    act, wide = mic.ACTIVATIONS.get(activation), _wide(x, out_dtype)
    if act is not None and wide is not None:
        r = (_native or _load()).linear(x, w, bias, residual, act, x_scale, w_scale, wide, return_preact, fast_sums)
        if r is not None:
            return r if return_preact else r[0]
    return_preact, fast_sums = _flag(return_preact, "return_preact"), _flag(fast_sums, "fast_sums")
    out_dtype = _layer_types(x, out_dtype, (x_scale, w_scale))
    act, dtype, device = _act(activation), x.dtype, x.device
    k = x.shape[-1] if x.dim() else 0
    m, ldx = _rows(x, k, "x")
    ldw = _weights(w, k, dtype, device, "w")
    n = w.shape[0]
    xs = _row_scale(x_scale, m, device)
    ws = 0 if w_scale is None else _vector(w_scale, n, torch.float32, device, "w_scale")
    bp = 0 if bias is None else _vector(bias, n, out_dtype, device, "bias")
    ldr = 0 if residual is None else _matrix(residual, m, n, out_dtype, device, "residual")
    h = _handle(device)
    shape = x.shape[:-1] + (n,)
    y = x.new_empty(shape, dtype=out_dtype)
    z = torch.empty_like(y) if return_preact else None
    fn = "mic_linear_forward_workspace" + ("_aligned" if _even((x, ldx), (w, ldw)) else "")
    wk, wkp, wkn = _workspace(fn, h, x, _CODE[dtype], m, n, k)
    _call("mic_linear_forward", h, _CODE[dtype], _CODE[out_dtype], act, fast_sums, m, n, k, x.data_ptr(), ldx, w.data_ptr(), ldw,
          xs, ws, bp, _ptr(residual), ldr, y.data_ptr(), n, _ptr(z), n, wkp, wkn)
    return (y, z) if return_preact else y


def linear_backward(dy, x, w, preact=None, activation="none", bias=False, need_dx=True, need_dw=True):
    """(dx, dw, dbias) of linear, from its inputs and preact (None without an activation).

    dbias is None unless bias is true, and dx and dw are where need_dx and
    need_dw are false (a first layer, frozen weights): what is None is not
    computed.  The residual's gradient is dy.
    """
    act = mic.ACTIVATIONS.get(activation)
    if act is not None:
        r = (_native or _load()).linear_backward(dy, x, w, preact, act, bias, need_dx, need_dw)
        if r is not None:
            return r
    bias, need_dx, need_dw = _flag(bias, "bias"), _flag(need_dx, "need_dx"), _flag(need_dw, "need_dw")
    _gpu(dy, "dy", (torch.float32, torch.bfloat16))
    act, dtype, device = _act(activation), dy.dtype, dy.device
    n = dy.shape[-1] if dy.dim() else 0
    m, lddy = _rows(dy, n, "dy")
    k = x.shape[-1] if x.dim() else 0
    ldx = _matrix(x, m, k, dtype, device, "x")
    ldw = _weights(w, k, dtype, device, "w")
    if w.shape[0] != n:
        raise ValueError("w has %d output features, dy %d" % (w.shape[0], n))
    if act and preact is None:
        raise ValueError("the gradient of activation %r needs preact" % activation)
    ldp = _matrix(preact, m, n, dtype, device, "preact") if act else 0
    h = _handle(device)
    dx = _empty(x.shape, x, dtype) if need_dx else None
    dw = _empty(w.shape, w, dtype) if need_dw else None
    dbias = dy.new_empty(n) if bias else None
    if _even((x, ldx), (w, ldw)) and (act or _even((dy, lddy))):
        wk, wkp, wkn = _workspace("mic_linear_backward_workspace_aligned", h, dy, _CODE[dtype], act, m, n, k)
    else:
        wk, wkp, wkn = _workspace("mic_linear_backward_workspace", h, dy, _CODE[dtype], m, n, k)
    _call("mic_linear_backward", h, _CODE[dtype], act, m, n, k, dy.data_ptr(), lddy, x.data_ptr(), ldx, w.data_ptr(),
          ldw, _ptr(preact) if act else 0, ldp, _ptr(dx), k, _ptr(dw), k, _ptr(dbias), wkp, wkn)
    return dx, dw, dbias


def gated_linear(x, w_gate, w_up, activation="silu", x_scale=None, w_gate_scale=None, w_up_scale=None,
                 out_dtype=None, return_products=False, fast_sums=False):
    """activation(x w_gate^T) * (x w_up^T); types, scales and fast_sums as linear's.

    return_products: (y, gate, up) with the two products, for
    gated_linear_backward.
    """
    act, wide = mic.ACTIVATIONS.get(activation), _wide(x, out_dtype)
    if act is not None and wide is not None:
        r = (_native or _load()).gated_linear(x, w_gate, w_up, act, x_scale, w_gate_scale, w_up_scale, wide,
                                              return_products, fast_sums)
        if r is not None:
            return r if return_products else r[0]
    return_products, fast_sums = _flag(return_products, "return_products"), _flag(fast_sums, "fast_sums")
    out_dtype = _layer_types(x, out_dtype, (x_scale, w_gate_scale, w_up_scale))
    act, dtype, device = _act(activation), x.dtype, x.device
    k = x.shape[-1] if x.dim() else 0
    m, ldx = _rows(x, k, "x")
    ldg = _weights(w_gate, k, dtype, device, "w_gate")
    ldu = _weights(w_up, k, dtype, device, "w_up")
    n = w_gate.shape[0]
    if w_up.shape[0] != n:
        raise ValueError("w_gate has %d output features, w_up %d" % (n, w_up.shape[0]))
    xs = _row_scale(x_scale, m, device)
    gs = 0 if w_gate_scale is None else _vector(w_gate_scale, n, torch.float32, device, "w_gate_scale")
    us = 0 if w_up_scale is None else _vector(w_up_scale, n, torch.float32, device, "w_up_scale")
    h = _handle(device)
    shape = x.shape[:-1] + (n,)
    y = x.new_empty(shape, dtype=out_dtype)
    gate = torch.empty_like(y) if return_products else None
    up = torch.empty_like(y) if return_products else None
    fn = "mic_gated_linear_forward_workspace" + ("_aligned" if _even((x, ldx), (w_gate, ldg), (w_up, ldu)) and ldg == ldu else "")
    wk, wkp, wkn = _workspace(fn, h, x, _CODE[dtype], m, n, k)
    _call("mic_gated_linear_forward", h, _CODE[dtype], _CODE[out_dtype], act, fast_sums, m, n, k, x.data_ptr(), ldx,
          w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu, xs, gs, us, y.data_ptr(), n, _ptr(gate), n, _ptr(up), n, wkp,
          wkn)
    return (y, gate, up) if return_products else y


def gated_linear_backward(dy, x, w_gate, w_up, gate, up, activation="silu", need_dx=True, need_dw=True):
    """(dx, dw_gate, dw_up) of gated_linear, from its inputs and two products.

    dx is None where need_dx is false, both weights' gradients where need_dw is:
    what is None is not computed.
    """
    act = mic.ACTIVATIONS.get(activation)
    if act is not None:
        r = (_native or _load()).gated_linear_backward(dy, x, w_gate, w_up, gate, up, act, need_dx, need_dw)
        if r is not None:
            return r
    need_dx, need_dw = _flag(need_dx, "need_dx"), _flag(need_dw, "need_dw")
    _gpu(dy, "dy", (torch.float32, torch.bfloat16))
    act, dtype, device = _act(activation), dy.dtype, dy.device
    n = dy.shape[-1] if dy.dim() else 0
    m, lddy = _rows(dy, n, "dy")
    k = x.shape[-1] if x.dim() else 0
    ldx = _matrix(x, m, k, dtype, device, "x")
    ldg = _weights(w_gate, k, dtype, device, "w_gate")
    ldu = _weights(w_up, k, dtype, device, "w_up")
    if w_gate.shape[0] != n or w_up.shape[0] != n:
        raise ValueError("w_gate and w_up have %d and %d output features, dy %d"
                         % (w_gate.shape[0], w_up.shape[0], n))
    ldgate = _matrix(gate, m, n, dtype, device, "gate")
    ldup = _matrix(up, m, n, dtype, device, "up")
    h = _handle(device)
    dx = _empty(x.shape, x, dtype) if need_dx else None
    dwg = _empty(w_gate.shape, w_gate, dtype) if need_dw else None
    dwu = _empty(w_up.shape, w_up, dtype) if need_dw else None
    fn = "mic_gated_linear_backward_workspace" + ("_aligned" if _even((x, ldx), (w_gate, ldg), (w_up, ldu)) and ldg == ldu else "")
    wk, wkp, wkn = _workspace(fn, h, dy, _CODE[dtype], m, n, k)
    _call("mic_gated_linear_backward", h, _CODE[dtype], act, m, n, k, dy.data_ptr(), lddy, x.data_ptr(), ldx,
          w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu, gate.data_ptr(), ldgate, up.data_ptr(), ldup, _ptr(dx), k, _ptr(dwg),
          k, _ptr(dwu), k, wkp, wkn)
    return dx, dwg, dwu
