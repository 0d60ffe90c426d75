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

from . import LlarError, _check, lib

__all__ = ["ACTIVATIONS", "linear", "linear_backward", "gated_ffn", "gated_ffn_backward"]

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_LINEAR, _LINEAR_BACKWARD, _GATED, _GATED_BACKWARD = 0, 1, 2, 3
_MATRIX_BYTES = 40  # llar_matrix: five 64-bit words

_codes = None
_space = {}


def _code(dtype) -> int:
    global _codes
    if _codes is None:
        import torch
        _codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    code = _codes.get(dtype)
    if code is None:
        raise TypeError("unsupported dtype %s (fp32, fp16, bf16 only)" % dtype)
    return code


def _act(name) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError("unknown activation %r (one of %s)" % (name, ", ".join(ACTIVATIONS)))
    return code


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


def _same(x, **others):
    if not x.is_cuda:
        raise LlarError(-4, "no GPU tensor: the operators run only on the HIP device")
    for name, t in others.items():
        if t is not None and (t.dtype != x.dtype or t.device != x.device):
            raise ValueError("%s must have x's type and device (%s, %s)" % (name, x.dtype, x.device))


def _expect(t, shape, what):
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (what, tuple(t.shape), tuple(shape)))


def _output(t, x, shape, what):
    import torch
    if t is None:
        return torch.empty(shape, dtype=x.dtype, device=x.device)
    _expect(t, shape, what)
    return t


def _raw_stream(device_index):
    """The current stream's handle, without building a torch stream object where torch offers that."""
    global _raw_stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _raw_stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(device_index)


def _call(fn, op, dims, dt, act, x, stream, inputs, outputs):
    """inputs, outputs: matrices (tensors of two dimensions), plain vectors (one dimension) or None, in the C
    call's order.  stream: a handle."""
    import torch
    words, args, unaligned = [], [], 0  # a matrix's place among the words goes into args as a negative number
    es = 4 if dt == 0 else 2
    for t in inputs:
        if t is None:
            args.append(None)
        elif t.dim() == 1:
            args.append(t.data_ptr())
        else:
            args.append(~(len(words) * 8))
            p, (rows, cols), (r, c) = t.data_ptr(), t.shape, t.stride()
            words += (p, rows, cols, r, c)
            width, line = (cols, r if rows > 1 else 0) if cols <= 1 or c == 1 else (rows, c)
            unaligned |= (p | (width | line) * es) & 15 | (line * es >= 1 << 23)
    for t in outputs:
        if t is None:
            args.append(None)
        elif t.dim() == 1:
            args.append(t.data_ptr())
        else:
            args.append(~(len(words) * 8))
            words += (t.data_ptr(), *t.shape, *t.stride())
    arr = (ctypes.c_int64 * len(words))(*words)
    at = ctypes.addressof(arr)
    args = [a if a is None or a >= 0 else at + ~a for a in args]
    key = (op, dt, unaligned) + dims
    need = _space.get(key)
    L = lib()
    if need is None:
        if len(_space) > 4096:
            _space.clear()
        need = _space[key] = L.llar_ffn_workspace(op, dims[0], dims[1], dims[2], dt, not unaligned)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    return getattr(L, fn)(*args, dt, act, ws.data_ptr() if need else None, need, stream)


def _on(x, stream, body):
    """Run body(stream handle) with x's device current and torch's allocations on the stream."""
    import torch
    if stream is None:
        at = x.get_device()
        if at == torch.cuda.current_device():
            return body(_raw_stream(at))
        with torch.cuda.device(at):
            return body(_raw_stream(at))
    if stream.device != x.device:
        raise ValueError("stream is on %s, x on %s" % (stream.device, x.device))
    with torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def linear(x, weight, bias=None, residual=None, activation="none", save=False, out=None, stream=None):
    """``activation(x @ weight.T + bias) + residual``.

    ``bias``: (n,) contiguous; ``residual``: the output's shape, rows contiguous; ``out`` may be ``residual``
    itself.  ``save``: also return the value before the activation, which ``linear_backward`` takes as ``pre``."""
    dt, act = _code(x.dtype), _act(activation)
    _same(x, weight=weight, bias=bias, residual=residual, out=out)
    x2 = _flat(x, "x")
    if weight.dim() != 2 or weight.shape[1] != x2.shape[1]:
        raise ValueError("weight has shape %s, expected (n, %d)" % (tuple(weight.shape), x2.shape[1]))
    n = weight.shape[0]
    shape = x.shape[:-1] + (n,)
    if bias is not None:
        _expect(bias, (n,), "bias")
        if n > 1 and bias.stride(0) != 1:
            raise ValueError("bias must be contiguous")
    if residual is not None:
        _expect(residual, shape, "residual")

    def body(s):
        y = _output(out, x, shape, "out")
        z = _output(None, x, shape, "pre") if save else None
        st = _call("llar_linear", _LINEAR, (x2.shape[0], n, x2.shape[1]), dt, act, x, s,
                   (x2, weight, bias, None if residual is None else _flat(residual, "residual")),
                   (_flat(y, "out"), _flat(z, "pre") if save else None))
        _check(st, "llar_linear")
        return (y, z) if save else y

    return _on(x, stream, body)


def linear_backward(dy, x, weight, pre=None, activation="none", input_grad=True, weight_grad=True, bias_grad=False,
                    stream=None):
    """Gradients (dx, dweight, dbias) of ``linear``; those not asked for are None.  The residual's gradient is
    ``dy`` itself.  ``pre``: the saved value before the activation (not needed without one)."""
    import torch
    dt, act = _code(x.dtype), _act(activation)
    _same(x, dy=dy, weight=weight, pre=pre)
    x2, dy2 = _flat(x, "x"), _flat(dy, "dy")
    if weight.dim() != 2 or weight.shape[1] != x2.shape[1]:
        raise ValueError("weight has shape %s, expected (n, %d)" % (tuple(weight.shape), x2.shape[1]))
    n = weight.shape[0]
    _expect(dy, x.shape[:-1] + (n,), "dy")
    if act:
        if pre is None:
            raise ValueError("pre, the value before the activation, is needed")
        _expect(pre, dy.shape, "pre")

    def body(s):
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if input_grad else None
        dw = torch.empty(weight.shape, dtype=x.dtype, device=x.device) if weight_grad else None
        db = torch.empty(n, dtype=x.dtype, device=x.device) if bias_grad else None
        st = _call("llar_linear_backward", _LINEAR_BACKWARD, (x2.shape[0], n, x2.shape[1]), dt, act, x, s,
                   (dy2, x2, weight, _flat(pre, "pre") if act else None),
                   (_flat(dx, "dx") if input_grad else None, dw, db))
        _check(st, "llar_linear_backward")
        return dx, dw, db

    return _on(x, stream, body)


def _gated_shapes(x2, w_gate, w_up):
    if w_gate.dim() != 2 or w_gate.shape[1] != x2.shape[1]:
        raise ValueError("w_gate has shape %s, expected (n, %d)" % (tuple(w_gate.shape), x2.shape[1]))
    _expect(w_up, w_gate.shape, "w_up")


def gated_ffn(x, w_gate, w_up, activation="silu", save=False, out=None, stream=None):
    """``activation(x @ w_gate.T) * (x @ w_up.T)`` in one kernel.  ``save``: also return both products, which
    ``gated_ffn_backward`` takes.  The weights have the same strides (two halves of one buffer, or two buffers)."""
    dt, act = _code(x.dtype), _act(activation)
    _same(x, w_gate=w_gate, w_up=w_up, out=out)
    x2 = _flat(x, "x")
    _gated_shapes(x2, w_gate, w_up)
    n = w_gate.shape[0]
    shape = x.shape[:-1] + (n,)

    def body(s):
        h = _output(out, x, shape, "out")
        g = _output(None, x, shape, "gate") if save else None
        u = _output(None, x, shape, "up") if save else None
        st = _call("llar_gated_ffn", _GATED, (x2.shape[0], n, x2.shape[1]), dt, act, x, s,
                   (x2, w_gate, w_up),
                   (_flat(h, "out"), _flat(g, "gate") if save else None, _flat(u, "up") if save else None))
        _check(st, "llar_gated_ffn")
        return (h, g, u) if save else h

    return _on(x, stream, body)


def gated_ffn_backward(dh, x, w_gate, w_up, gate, up, activation="silu", input_grad=True, weight_grad=True,
                       stream=None):
    """Gradients (dx, dw_gate, dw_up) of ``gated_ffn`` from the products it saved; those not asked for are None."""
    import torch
    dt, act = _code(x.dtype), _act(activation)
    _same(x, dh=dh, w_gate=w_gate, w_up=w_up, gate=gate, up=up)
    x2 = _flat(x, "x")
    _gated_shapes(x2, w_gate, w_up)
    n = w_gate.shape[0]
    for t, what in ((dh, "dh"), (gate, "gate"), (up, "up")):
        _expect(t, x.shape[:-1] + (n,), what)

    def body(s):
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if input_grad else None
        dwg = torch.empty(w_gate.shape, dtype=x.dtype, device=x.device) if weight_grad else None
        dwu = torch.empty(w_gate.shape, dtype=x.dtype, device=x.device) if weight_grad else None
        st = _call("llar_gated_ffn_backward", _GATED_BACKWARD, (x2.shape[0], n, x2.shape[1]), dt, act, x, s,
                   (_flat(dh, "dh"), x2, w_gate, w_up, _flat(gate, "gate"), _flat(up, "up")),
                   (_flat(dx, "dx") if input_grad else None, dwg, dwu))
        _check(st, "llar_gated_ffn_backward")
        return dx, dwg, dwu

    return _on(x, stream, body)
