"""Feed-forward operators of a tensor-parallel layer (torch tensors in, torch
tensors out): the row-parallel matrix product with its epilogue, the gated
block's column-parallel products, and both backward passes.  The kernels are
the library's (``include/llar.h``); this module checks and marshals arguments.

Tensors are fp32, fp16 or bf16 device tensors of one type.  ``x`` and the other
activations have shape (..., width), with leading dimensions that can be viewed
as one; weights are (n, k).  A matrix may be strided along one axis (a slice of
a wider buffer, a transposed view, an expanded row).  Nothing is recorded for
autograd: ``linear_backward`` and ``gated_ffn_backward`` are the gradients.

``stream`` is a torch stream (default: the current one of x's device).  Outputs
and workspace come from torch's allocator on that stream; inputs made on another
stream have to be ordered before it by the caller, as for any torch operator.
"""
from __future__ import annotations

import ctypes

from . import LlarError, lib

__all__ = ["ACTIVATIONS", "linear", "linear_backward", "gated_ffn", "gated_ffn_backward"]

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_LINEAR, _LINEAR_BACKWARD, _GATED, _GATED_BACKWARD = 0, 1, 2, 3
_words = [ctypes.c_int64 * n for n in range(51)]  # a llar_matrix is five 64-bit words

_torch = _codes = _raw_stream = None
_fn = {}
_space = {}


def _setup():
    """What a call needs of torch and the library, looked up once."""
    global _torch, _codes, _raw_stream
    import torch
    _codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    # the current stream's handle, without building a stream object where torch offers that
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _raw_stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
    L = lib()
    for op, name in enumerate(("llar_linear", "llar_linear_backward", "llar_gated_ffn", "llar_gated_ffn_backward")):
        _fn[op] = (getattr(L, name), name)
    _torch = torch


def _type_and_act(x, activation):
    if _torch is None:
        _setup()
    dt, act = _codes.get(x.dtype), ACTIVATIONS.get(activation)
    if dt is None:
        raise TypeError("unsupported dtype %s (fp32, fp16, bf16 only)" % x.dtype)
    if act is None:
        raise ValueError("unknown activation %r (one of %s)" % (activation, ", ".join(ACTIVATIONS)))
    if not x.is_cuda:
        raise LlarError(-4, "no GPU tensor: the operators run only on the HIP device")
    return dt, act


def _flat(t, what):
    """A (..., width) tensor as a matrix that shares its memory."""
    if t.dim() == 2:
        return t
    if t.dim() == 0:
        raise ValueError("%s needs at least one dimension" % what)
    try:
        return t.view(-1, t.shape[-1]) if t.numel() else t.reshape(t.shape[:-1].numel(), t.shape[-1])
    except RuntimeError:
        raise ValueError("%s: the leading dimensions cannot be viewed as one; make it contiguous" % what) from None


def _like(x, t, shape, what):
    """t has x's type and device, and the shape."""
    if t.dtype != x.dtype or t.get_device() != x.get_device():
        raise ValueError("%s must have x's type and device (%s, %s)" % (what, x.dtype, x.device))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (what, tuple(t.shape), tuple(shape)))


def _weight(x, k, w, what):
    if w.dim() != 2 or w.shape[1] != k:
        raise ValueError("%s has shape %s, expected (n, %d)" % (what, tuple(w.shape), k))
    _like(x, w, w.shape, what)
    return w.shape[0]


def _call(op, dims, dt, act, x, stream, inputs, outputs):
    """inputs, outputs: matrices (tensors of two dimensions), plain vectors (one dimension) or None, in the C
    call's order, of which the inputs open with (dy,) x, weight.  stream: a handle."""
    words, args = [], []  # a matrix's place among the words goes into args as a negative number
    es = 4 if dt == 0 else 2
    loose = columns = 0
    for i, t in enumerate(inputs):
        if t is None:
            args.append(None)
        elif t.dim() == 1:
            args.append(t.data_ptr())
        else:
            args.append(~(len(words) * 8))
            p, (rows, cols), (r, c) = t.data_ptr(), t.shape, t.stride()
            words += (p, rows, cols, r, c)
            if cols <= 1 or c == 1:
                width, line = cols, r if rows > 1 else 0
            else:
                width, line = rows, c
                columns |= 1 << i
            if (p | (width | line) * es) & 15 or line * es >= 1 << 23:
                loose = 1
    for t in outputs:
        if t is None:
            args.append(None)
        elif t.dim() == 1:
            args.append(t.data_ptr())
        else:
            args.append(~(len(words) * 8))
            words += (t.data_ptr(), *t.shape, *t.stride())
    arr = _words[len(words)](*words)
    at = ctypes.addressof(arr)
    key = (op, dt, dims, loose, columns)
    need = _space.get(key)
    if need is None:
        if len(_space) > 4096:
            _space.clear()
        if op & 1:  # a backward pass: (dy, x, weight)
            columns = (columns >> 1 & 3) | (columns & 1) << 2
        need = _space[key] = lib().llar_ffn_workspace(op, *dims, dt, loose | (columns & 7) << 1)
    ws = x.new_empty(need, dtype=_torch.uint8) if need else None
    fn, name = _fn[op]
    st = fn(*[a if a is None or a >= 0 else at + ~a for a in args], dt, act, ws.data_ptr() if need else None, need,
            stream)
    if st < 0:
        raise LlarError(st, name)


def _elsewhere(x, stream, body):
    """Runs body, which works on x's device's current stream, where device or stream are others."""
    if stream is None:
        with _torch.cuda.device(x.device):
            return body()
    if stream.device != x.device:
        raise ValueError("stream is on %s, x on %s" % (stream.device, x.device))
    with _torch.cuda.stream(stream):
        return body()


def linear(x, weight, bias=None, residual=None, activation="none", save=False, out=None, stream=None):
    """``activation(x @ weight.T + bias) + residual``.

    ``bias``: (n,) contiguous; ``residual``: the output's shape, rows contiguous; ``out`` may be ``residual``
    itself.  ``save``: also return the value before the activation, which ``linear_backward`` takes as ``pre``."""
    dt, act = _type_and_act(x, activation)
    at = x.get_device()
    if stream is not None or at != _torch.cuda.current_device():
        return _elsewhere(x, stream, lambda: linear(x, weight, bias, residual, activation, save, out))
    x2 = _flat(x, "x")
    m, k = x2.shape
    n = _weight(x, k, weight, "weight")
    shape = x.shape[:-1] + (n,)
    if bias is not None:
        _like(x, bias, (n,), "bias")
        if n > 1 and bias.stride(0) != 1:
            raise ValueError("bias must be contiguous")
    if residual is not None:
        _like(x, residual, shape, "residual")
        residual = _flat(residual, "residual")
    if out is None:
        out = x.new_empty(shape)
    else:
        _like(x, out, shape, "out")
    pre = x.new_empty(shape) if save else None
    _call(_LINEAR, (m, n, k), dt, act, x, _raw_stream(at), (x2, weight, bias, residual),
          (_flat(out, "out"), _flat(pre, "pre") if save else None))
    return (out, pre) if save else out


def linear_backward(dy, x, weight, pre=None, activation="none", input_grad=True, weight_grad=True, bias_grad=False,
                    stream=None):
    """Gradients (dx, dweight, dbias) of ``linear``; those not asked for are None.  The residual's gradient is
    ``dy`` itself.  ``pre``: the saved value before the activation (not needed without one)."""
    dt, act = _type_and_act(x, activation)
    at = x.get_device()
    if stream is not None or at != _torch.cuda.current_device():
        return _elsewhere(x, stream, lambda: linear_backward(dy, x, weight, pre, activation, input_grad, weight_grad,
                                                             bias_grad))
    x2 = _flat(x, "x")
    m, k = x2.shape
    n = _weight(x, k, weight, "weight")
    shape = x.shape[:-1] + (n,)
    _like(x, dy, shape, "dy")
    if act:
        if pre is None:
            raise ValueError("pre, the value before the activation, is needed")
        _like(x, pre, shape, "pre")
        pre = _flat(pre, "pre")
    else:
        pre = None
    dx = x.new_empty(x.shape) if input_grad else None
    dw = x.new_empty((n, k)) if weight_grad else None
    db = x.new_empty((n,)) if bias_grad else None
    _call(_LINEAR_BACKWARD, (m, n, k), dt, act, x, _raw_stream(at), (_flat(dy, "dy"), x2, weight, pre),
          (_flat(dx, "dx") if input_grad else None, dw, db))
    return dx, dw, db


def gated_ffn(x, w_gate, w_up, activation="silu", save=False, out=None, stream=None):
    """``activation(x @ w_gate.T) * (x @ w_up.T)`` in one kernel.  ``save``: also return both products, which
    ``gated_ffn_backward`` takes.  The weights have the same strides (two halves of one buffer, or two buffers)."""
    dt, act = _type_and_act(x, activation)
    at = x.get_device()
    if stream is not None or at != _torch.cuda.current_device():
        return _elsewhere(x, stream, lambda: gated_ffn(x, w_gate, w_up, activation, save, out))
    x2 = _flat(x, "x")
    m, k = x2.shape
    n = _weight(x, k, w_gate, "w_gate")
    _like(x, w_up, w_gate.shape, "w_up")
    shape = x.shape[:-1] + (n,)
    if out is None:
        out = x.new_empty(shape)
    else:
        _like(x, out, shape, "out")
    gate, up = (x.new_empty(shape), x.new_empty(shape)) if save else (None, None)
    _call(_GATED, (m, n, k), dt, act, x, _raw_stream(at), (x2, w_gate, w_up),
          (_flat(out, "out"), _flat(gate, "gate") if save else None, _flat(up, "up") if save else None))
    return (out, gate, up) if save else out


def gated_ffn_backward(dh, x, w_gate, w_up, gate, up, activation="silu", input_grad=True, weight_grad=True,
                       stream=None):
    """Gradients (dx, dw_gate, dw_up) of ``gated_ffn`` from the products it saved; those not asked for are None."""
    dt, act = _type_and_act(x, activation)
    at = x.get_device()
    if stream is not None or at != _torch.cuda.current_device():
        return _elsewhere(x, stream, lambda: gated_ffn_backward(dh, x, w_gate, w_up, gate, up, activation, input_grad,
                                                                weight_grad))
    x2 = _flat(x, "x")
    m, k = x2.shape
    n = _weight(x, k, w_gate, "w_gate")
    _like(x, w_up, w_gate.shape, "w_up")
    shape = x.shape[:-1] + (n,)
    _like(x, dh, shape, "dh")
    _like(x, gate, shape, "gate")
    _like(x, up, shape, "up")
    dx = x.new_empty(x.shape) if input_grad else None
    dwg, dwu = (x.new_empty((n, k)), x.new_empty((n, k))) if weight_grad else (None, None)
    _call(_GATED_BACKWARD, (m, n, k), dt, act, x, _raw_stream(at),
          (_flat(dh, "dh"), x2, w_gate, w_up, _flat(gate, "gate"), _flat(up, "up")),
          (_flat(dx, "dx") if input_grad else None, dwg, dwu))
    return dx, dwg, dwu
