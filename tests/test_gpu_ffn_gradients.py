"""Incoming gradients as autograd hands them over: transposed views, values
repeated along one axis or both (the gradient of a sum), slices with a step."""
import pytest
import torch

import message_allreduce_amd as llar
from test_gpu_ffn import ACTS, DTYPES, EPS, Draw, check, ids, linear_backward_case, mm64

pytestmark = pytest.mark.gpu

SIZES = [(1, 40, 64), (7, 33, 50), (16, 264, 520), (72, 136, 88), (515, 72, 40), (300, 1100, 264)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dyl", ["col", "colpad"])
def test_transposed_gradients(dyl, act, dtype):
    for size in SIZES:
        linear_backward_case(*size, dtype, act, dyl=dyl)
        linear_backward_case(*size, dtype, act, dyl=dyl, bias=False, xl="col", wl="col")


def repeated(d, m, n, how):
    if how == "one value":
        return d(1, 1).expand(m, n)
    if how == "one row":
        return d(1, n).expand(m, n)
    if how == "one column":
        return d(m, 1).expand(m, n)
    if how == "transposed":
        return d(n, m).t()
    return d(2 * m, 3 * n)[::2, 1::3]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("how", ["one value", "one row", "one column", "transposed", "step"])
def test_gradients_of_any_strides_give_what_their_copies_give(how, dtype):
    for m, n, k in SIZES:
        for act in ("none", "silu"):
            d = Draw(m * n + k, dtype)
            x, w, wu, z, g, u = d(m, k), d(n, k), d(n, k), d(m, n), d(m, n), d(m, n)
            dy = repeated(d, m, n, how)
            pre = None if act == "none" else z
            for bias in ((True,) if how == "transposed" else (False, True)):
                got = llar.linear_backward(dy, x, w, pre, activation=act, bias_grad=bias)
                want = llar.linear_backward(dy.contiguous(), x, w, pre, activation=act, bias_grad=bias)
                if how == "one column" and act == "none" and not bias:
                    # read where it lies, as the column-contiguous matrix it is: the sums' order may differ
                    Y, X, W = dy.double(), x.double(), w.double()
                    check(got[0], mm64(Y, W), (n + 16) * EPS * mm64(Y.abs(), W.abs()), "dx")
                    check(got[1], mm64(Y.t(), X), (m + 16) * EPS * mm64(Y.t().abs(), X.abs()), "dw")
                    continue
                for a, b in zip(got, want):
                    assert (a is None and b is None) or torch.equal(a, b), (m, n, k, act, bias)
            for a, b in zip(llar.gated_ffn_backward(dy, x, w, wu, g, u, activation=act),
                            llar.gated_ffn_backward(dy.contiguous(), x, w, wu, g, u, activation=act)):
                assert torch.equal(a, b), (m, n, k, act)


def test_leading_dimensions_and_a_whole_sum():
    d = Draw(3, torch.bfloat16)
    x, w = d(6, 64), d(40, 64)
    y, z = llar.linear(x.view(2, 3, 64), w, activation="gelu", save=True)
    one = torch.ones((), dtype=torch.bfloat16, device="cuda").expand(2, 3, 40)  # the gradient of y.sum()
    got = llar.linear_backward(one, x.view(2, 3, 64), w, z, activation="gelu", bias_grad=True)
    want = llar.linear_backward(one.contiguous(), x.view(2, 3, 64), w, z, activation="gelu", bias_grad=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals():
    d = Draw(1, torch.float32)
    x, w = d(4, 64), d(32, 64)
    long = torch.zeros(1, 1, device="cuda").expand(2, 1 << 21)  # its copy's rows would be longer than a line may be
    wide = torch.zeros(1, 1, device="cuda").expand(1 << 21, 64)
    for bad in (lambda: llar.linear_backward(long, x[:2], wide),
                lambda: llar.linear_backward(d(32, 4).t(), x, w, d(32, 4).t(), activation="silu"),  # pre's rows
                lambda: llar.gated_ffn_backward(d(4, 32), x, w, w, d(32, 4).t(), d(4, 32)),
                lambda: llar.gated_ffn_backward(d(4, 32), x, w, w, d(4, 32), d(32, 4).t())):
        with pytest.raises(llar.LlarError):
            bad()
