"""Feed-forward operators of a tensor-parallel layer (torch tensors in, torch
tensors out): the row-parallel matrix product with its epilogue, the gated
block's column-parallel products, and both backward passes.  The kernels are
the library's (``include/llar.h``); this module checks and marshals arguments.

Tensors are fp32, fp16 or bf16 device tensors of one type.  ``x`` and the other
activations have shape (..., width), with leading dimensions that can be viewed
as one; weights are (n, k).  A matrix may be strided along one axis (a slice of
a wider buffer, a transposed view, an expanded row), the incoming gradients
``dy`` and ``dh`` along both (the gradient of a sum).  Nothing is recorded for
autograd: ``linear_backward`` and ``gated_ffn_backward`` are the gradients.

``stream`` is a torch stream (default: the current one of x's device).  Outputs
and workspace come from torch's allocator on that stream; inputs made on another
stream have to be ordered before it by the caller, as for any torch operator.
"""
from __future__ import annotations

from . import LlarError, lib

__all__ = ["ACTIVATIONS", "linear", "linear_backward", "gated_ffn", "gated_ffn_backward"]

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_native = None


def _setup():
    """Load the binding (csrc/llar_py.c) and hand it what it needs of torch, once."""
    global _native
    import torch
    lib()  # raises if the library is not built
    try:
        from . import _llar_py as native
    except ImportError as e:
        raise LlarError(-4, "_llar_py is not built (run __graft_entry__.build(); it needs a C compiler and "
                        "Python.h): %s" % e) from None
    # the current device and stream's handle, without building objects where torch offers that
    device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    native.setup(torch.float32, torch.float16, torch.bfloat16, torch.uint8, device, stream, LlarError)
    _native = native
    return native


def _elsewhere(x, stream, body, *args):
    """body(*args), which works on the current device and stream, on x's device or the stream given."""
    import torch
    if stream is None:
        with torch.cuda.device(x.device):
            return body(*args)
    if stream.device != x.device:
        raise ValueError("stream is on %s, x on %s" % (stream.device, x.device))
    with torch.cuda.stream(stream):
        return body(*args)


def linear(x, weight, bias=None, residual=None, activation="none", save=False, out=None, stream=None):
    """``activation(x @ weight.T + bias) + residual``.

    ``bias``: (n,) contiguous; ``residual``: the output's shape, rows contiguous; ``out`` may be ``residual``
    itself.  ``save``: also return the value before the activation, which ``linear_backward`` takes as ``pre``."""
    f = (_native or _setup()).linear
    args = (x, weight, bias, residual, activation, save, out)
    r = NotImplemented if stream is not None else f(*args)
    return r if r is not NotImplemented else _elsewhere(x, stream, f, *args)


def linear_backward(dy, x, weight, pre=None, activation="none", input_grad=True, weight_grad=True, bias_grad=False,
                    stream=None):
    """Gradients (dx, dweight, dbias) of ``linear``; those not asked for are None.  The residual's gradient is
    ``dy`` itself.  ``pre``: the saved value before the activation (not needed without one)."""
    f = (_native or _setup()).linear_backward
    args = (dy, x, weight, pre, activation, input_grad, weight_grad, bias_grad)
    r = NotImplemented if stream is not None else f(*args)
    return r if r is not NotImplemented else _elsewhere(x, stream, f, *args)


def gated_ffn(x, w_gate, w_up, activation="silu", save=False, out=None, stream=None):
    """``activation(x @ w_gate.T) * (x @ w_up.T)`` in one kernel.  ``save``: also return both products, which
    ``gated_ffn_backward`` takes.  The weights have the same strides (two halves of one buffer, or two buffers)."""
    f = (_native or _setup()).gated_ffn
    args = (x, w_gate, w_up, activation, save, out)
    r = NotImplemented if stream is not None else f(*args)
    return r if r is not NotImplemented else _elsewhere(x, stream, f, *args)


def gated_ffn_backward(dh, x, w_gate, w_up, gate, up, activation="silu", input_grad=True, weight_grad=True,
                       stream=None):
    """Gradients (dx, dw_gate, dw_up) of ``gated_ffn`` from the products it saved; those not asked for are None."""
    f = (_native or _setup()).gated_ffn_backward
    args = (dh, x, w_gate, w_up, gate, up, activation, input_grad, weight_grad)
    r = NotImplemented if stream is not None else f(*args)
    return r if r is not NotImplemented else _elsewhere(x, stream, f, *args)
