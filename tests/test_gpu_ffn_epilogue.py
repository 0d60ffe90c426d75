"""The product's epilogue with every order of its operands: bias, residual,
activation and kept pre-activation over weights that lie n x k and k x n, whole
and odd, against binary64 with the tolerances of test_gpu_ffn.py."""
import pytest
import torch

import message_allreduce_amd as llar
from test_gpu_ffn import DTYPES, EPS, Draw, act64, check, ids, linear_case, mm64

pytestmark = pytest.mark.gpu

# rows on both sides of 16, and products that want each tile shape, whole in k and split between workgroups
SIZES = [(5, 72, 96), (16, 520, 1000), (17, 40, 40), (17, 40, 200), (17, 4100, 2000), (40, 72, 64), (100, 1096, 1000),
         (200, 2000, 4000), (500, 4100, 40), (500, 4104, 200), (1000, 2000, 504), (2000, 2000, 200), (2000, 4100, 40),
         (3000, 40, 2000), (3000, 4104, 640)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("wl", ["row", "off", "col", "colpad"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_residual_with_every_order_of_the_weights(size, wl, dtype):
    for bias in (False, True):
        linear_case(*size, dtype, "none", bias, True, wl=wl)
    linear_case(*size, dtype, "none", False, True, save=True, wl=wl)
    linear_case(*size, dtype, "gelu", True, True, save=size[0] < 100, wl=wl, xl="col")


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("act", ["relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("wl", ["off", "col", "colpad"])
def test_epilogue_parts_with_every_order_of_the_weights(wl, act, dtype):
    for bias in (False, True):
        for residual in (False, True):
            for m, n, k in ((9, 72, 136), (40, 72, 64), (300, 264, 136), (45, 71, 33)):
                linear_case(m, n, k, dtype, act, bias, residual, save=bias != residual, wl=wl)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("wl", ["row", "col"])
@pytest.mark.parametrize("size", [(40, 136, 72), (300, 264, 136), (3000, 4104, 576)], ids=str)
def test_residuals_of_every_layout(size, wl, dtype):
    """Rows apart, unaligned, repeated, and the output itself."""
    m, n, k = size
    d = Draw(m + n, dtype)
    x, w, b = d(m, k), d(n, k, wl, k ** -0.5), d(1, n)[0]
    X, W = x.double(), w.double()
    want, A = mm64(X, W.t()), mm64(X.abs(), W.t().abs())
    for rl in ("row", "pad", "off", "one", "out"):
        for act in ("none", "silu"):
            r = d(1, n).expand(m, n) if rl == "one" else d(m, n, "row" if rl == "out" else rl)
            z, zerr = want + b.double(), (k + 16) * EPS * (A + b.double().abs())
            y64 = act64(z, act)
            err = zerr if act == "none" else 1.2 * zerr + 16 * EPS * y64.abs()
            r64 = r.double()
            y = llar.linear(x, w, b, r, activation=act, out=r if rl == "out" else None)
            check(y, y64 + r64, err + EPS * ((y64 + r64).abs() + r64.abs()), "residual %s, %s" % (rl, act))
