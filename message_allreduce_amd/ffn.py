"""Feed-forward operators of a tensor-parallel layer (torch tensors in, torch
tensors out): the row-parallel matrix product with its epilogue, the gated
block's column-parallel products, and both backward passes; for serving, the
products with 8-bit weights and the mixture-of-experts layer.  The kernels are
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

__all__ = ["ACTIVATIONS", "linear", "linear_backward", "gated_ffn", "gated_ffn_backward", "quantize_rows",
           "linear_int8", "gated_ffn_int8", "moe_route", "moe_ffn"]

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
    native.setup(torch.float32, torch.float16, torch.bfloat16, torch.uint8, torch.int8, torch.int32, torch.int64, device,
                 stream, LlarError)
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


# ---- products of 8-bit whole numbers -----------------------------------------------

def quantize_rows(x, stream=None):
    """(q, scale): ``scale`` (float32) the largest magnitude of each row of x (..., k) over 127, ``q`` (int8, x's
    shape) the nearest whole numbers to ``x / scale``, ties to even.  Tokens are quantised so before
    ``linear_int8``, and a weight's output channels, which are its rows.  A row of zeros, or of magnitudes below 2^-143,
    has scale 0; one with an infinity or a NaN has scale NaN, and so do the products it enters."""
    f = (_native or _setup()).quantize_rows
    r = NotImplemented if stream is not None else f(x)
    return r if r is not NotImplemented else _elsewhere(x, stream, f, x)


def linear_int8(x, weight, w_scale, x_scale=None, bias=None, residual=None, activation="none", dtype=None, out=None,
                stream=None):
    """``activation(x_scale * w_scale * (x @ weight.T) + bias) + residual`` with exact whole-number sums.

    ``weight`` (n, k) int8 with contiguous rows and ``w_scale`` (n,) float32, as ``quantize_rows`` makes them.  x:
    (..., k) int8 with ``x_scale`` (...,), or fp32, fp16 or bf16 without it, which the call quantises the same way.
    ``dtype``: the output's type, bias's and residual's (x's own, or bf16 for int8 x).  k is at most 2^17 - 1."""
    f = (_native or _setup()).linear_int8
    args = (x, weight, w_scale, x_scale, bias, residual, activation, dtype, out)
    r = NotImplemented if stream is not None else f(*args)
    return r if r is not NotImplemented else _elsewhere(x, stream, f, *args)


def gated_ffn_int8(x, w_gate, w_up, gate_scale, up_scale, x_scale=None, activation="silu", dtype=None, out=None,
                   stream=None):
    """``activation(g) * u`` of the two 8-bit products g and u of x with ``w_gate`` and ``w_up``, in one kernel (and
    one that quantises x, if it is not int8).  Arguments as ``linear_int8``'s and ``gated_ffn``'s."""
    f = (_native or _setup()).gated_ffn_int8
    args = (x, w_gate, w_up, gate_scale, up_scale, x_scale, activation, dtype, out)
    r = NotImplemented if stream is not None else f(*args)
    return r if r is not NotImplemented else _elsewhere(x, stream, f, *args)


# ---- mixture of experts for a few tokens --------------------------------------------

def moe_route(x, router, top_k, scoring="softmax", normalize=True, stream=None):
    """(weights, experts), (..., top_k) each: for every token of x (..., k) the ``top_k`` rows of ``router``
    (experts, k) with the largest products, in falling order, of equals the lowest number first (int32), and their
    ``scoring`` (float32): "softmax" over all experts, or each product's "sigmoid"; ``normalize``: divided by their
    sum.  The products are summed in binary64; two that differ by less than its rounding may be taken in
    either order, which may be another one with more tokens."""
    if scoring not in ("softmax", "sigmoid"):
        raise ValueError("unknown scoring %r (softmax or sigmoid)" % (scoring,))
    f = (_native or _setup()).moe_route
    args = (x, router, top_k, scoring == "sigmoid", normalize)
    r = NotImplemented if stream is not None else f(*args)
    return r if r is not NotImplemented else _elsewhere(x, stream, f, *args)


def moe_ffn(x, experts, weights, w_gate, w_up, w_down, activation="silu", residual=None, gate_scale=None, up_scale=None,
            down_scale=None, out=None, stream=None):
    """The sum over a token's experts of ``weight * (activation(x @ wg.T) * (x @ wu.T)) @ wd.T``, + ``residual``, in
    two kernels.

    x (..., k); ``experts`` (..., top_k) int32 or int64 and ``weights`` float32, contiguous, as ``moe_route`` returns
    them; ``w_gate`` and ``w_up`` (E, n, k) with the same strides, ``w_down`` (E, outputs, n), contiguous along their
    last axis.  A number outside 0 .. E - 1 (an expert of another rank, a padded token) adds nothing; the output is
    then a partial one for the AllReduce.  With ``gate_scale``, ``up_scale`` (E, n) and ``down_scale`` (E, outputs),
    float32, the weights are int8; x and the inner rows are quantised as ``quantize_rows`` does.

    The inner values of fp16 end at 65504 and are infinite beyond (``gated_ffn``'s do too); those of bf16, fp32 and
    int8 weights have float32's range.  Made for a step's tokens: a chosen expert's weights are read once for every 64
    of them, so 65 take as long as 64 and 1, and 128 twice as long as 64."""
    f = (_native or _setup()).moe_ffn
    args = (x, experts, weights, w_gate, w_up, w_down, gate_scale, up_scale, down_scale, activation, residual, out)
    r = NotImplemented if stream is not None else f(*args)
    return r if r is not NotImplemented else _elsewhere(x, stream, f, *args)
