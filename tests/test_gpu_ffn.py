"""The feed-forward operators against their formulas in binary64.

Tolerances.  With u the I/O type's unit roundoff (2^-24, 2^-11, 2^-8) and A the
same sum of products taken over absolute values, a sum of k binary32 terms is
off by at most (k + 16) 2^-23 A; an activation of slope at most 1.2 passes that
on, and is itself evaluated to 16 roundings of binary32; the output rounds
once.  In the backward passes the gradient that both products read is rounded
to the I/O type first: another u A.  fp16 outputs round absolutely below 2^-14
(2^-25), and its rounded gradients carry that into the sums.
"""
import math

import pytest
import torch

import message_allreduce_amd as llar

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
EPS = 2.0 ** -23


def ids(v):
    return str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None


def act64(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def slope64(z, act):
    if act == "none":
        return torch.ones_like(z)
    z = z.clone().requires_grad_(True)
    return torch.autograd.grad(act64(z, act).sum(), z)[0]


def mm64(a, b):
    return torch.mm(a.contiguous(), b.contiguous())


class Draw:
    def __init__(self, seed, dtype):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.dtype = dtype

    def __call__(self, rows, cols, layout="row", scale=1.0):
        """A rows x cols matrix: "row" (dense), "pad" (rows of a wider buffer), "off" (rows at an odd element),
        "col" (a transposed view), "colpad" (transposed, from a wider buffer)."""
        def t(r, c):
            return torch.empty(r, c, dtype=self.dtype, device="cuda").normal_(0, scale, generator=self.g)
        if layout == "row":
            return t(rows, cols)
        if layout == "pad":
            return t(rows, cols + 8)[:, :cols]
        if layout == "off":
            return t(rows, cols + 3)[:, 1:cols + 1]
        if layout == "col":
            return t(cols, rows).t()
        return t(cols, rows + 8)[:, :rows].t()


def check(got, want, err, what):
    """err: the bound on the unrounded result."""
    u, tiny = U[got.dtype], TINY[got.dtype]
    g = got.double()
    assert g.shape == want.shape, what
    tol = 1.01 * u * want.abs() + 1.02 * err + tiny
    bad = ~((g - want).abs() <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d outside; first at %s: %r, expected %r, allowed %r"
                             % (what, int(bad.sum()), bad.numel(), i, g[i].item(), want[i].item(), tol[i].item()))


def linear_case(m, n, k, dtype, act="none", bias=False, residual=False, save=False, xl="row", wl="row", seed=0):
    d = Draw(seed * 7919 + m * 31 + n * 17 + k, dtype)
    x, w = d(m, k, xl), d(n, k, wl, k ** -0.5 if k else 1.0)
    b = d(1, n)[0] if bias else None
    r = d(m, n) if residual else None
    y = llar.linear(x, w, b, r, activation=act, save=save)
    y, z = y if save else (y, None)
    X, W = x.double(), w.double()
    want_z, A = mm64(X, W.t()), mm64(X.abs(), W.t().abs())
    if bias:
        want_z, A = want_z + b.double(), A + b.double().abs()
    err = (k + 16) * EPS * A
    if save:
        check(z, want_z, err, "pre")
    want = act64(want_z, act)
    err = 1.2 * err + 16 * EPS * want.abs()
    if residual:
        want, err = want + r.double(), err + EPS * (want.abs() + r.double().abs())
    check(y, want, err, "linear %s" % ((m, n, k, dtype, act, xl, wl),))


SIZES = [(1, 1, 1), (1, 512, 512), (1, 77, 130), (2, 64, 8), (3, 200, 96), (16, 64, 64), (17, 33, 65), (31, 129, 72),
         (64, 64, 2048), (65, 640, 320), (128, 128, 128), (200, 513, 257), (257, 256, 64), (300, 264, 1000)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_linear_sizes(size, dtype):
    linear_case(*size, dtype)
    linear_case(*size, dtype, act="gelu", bias=True, residual=True, save=True, seed=1)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("xl", ["row", "pad", "off", "col", "colpad"])
@pytest.mark.parametrize("wl", ["row", "pad", "off", "col", "colpad"])
def test_linear_layouts(xl, wl, dtype):
    for size in ((72, 136, 96), (33, 71, 45), (1, 40, 64), (9, 264, 520)):
        linear_case(*size, dtype, bias=True, xl=xl, wl=wl)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("act", ACTS)
def test_linear_epilogues(act, dtype):
    for bias in (False, True):
        for residual in (False, True):
            linear_case(40, 72, 64, dtype, act, bias, residual, save=bias)
            linear_case(4, 72, 1024, dtype, act, bias, residual, save=bias)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("size", [(2048, 2304, 512), (4096, 4096, 128), (1000, 4104, 264), (512, 512, 8192), (48, 8192, 1024)], ids=str)
def test_linear_large(size, dtype):
    linear_case(*size, dtype, act="silu", bias=True, residual=True)
    linear_case(*size, dtype, wl="col", xl="col")


def linear_backward_case(m, n, k, dtype, act, xl="row", wl="row", dyl="row", bias=True, seed=0):
    d = Draw(seed * 104729 + m * 13 + n * 7 + k, dtype)
    x, w, dy = d(m, k, xl), d(n, k, wl, k ** -0.5 if k else 1.0), d(m, n, dyl)
    z = d(m, n) if act != "none" else None
    dx, dw, db = llar.linear_backward(dy, x, w, z, activation=act, bias_grad=bias)
    u = U[dtype] if act != "none" else 0.0
    tiny = TINY[dtype] if act != "none" else 0.0
    dz = dy.double() if z is None else dy.double() * slope64(z.double(), act)
    # the slope is off by 16 roundings of binary32, of terms up to |z|
    dzerr = 0 * dz if z is None else 20 * EPS * dy.double().abs() * (1 + z.double().abs())
    e = dzerr + (u * 1.01 + 0.0) * dz.abs() + tiny
    X, W = x.double(), w.double()
    check(dx, mm64(dz, W), mm64(e, W.abs()) + (n + 16) * EPS * mm64(dz.abs(), W.abs()), "dx")
    check(dw, mm64(dz.t(), X), mm64(e.t(), X.abs()) + (m + 16) * EPS * mm64(dz.t().abs(), X.abs()), "dw")
    if bias:
        check(db, dz.sum(0), (dzerr + (m + 16) * EPS * dz.abs()).sum(0), "db")
    else:
        assert db is None


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", [(1, 64, 64), (7, 33, 50), (64, 128, 96), (130, 257, 264), (515, 72, 40)], ids=str)
def test_linear_backward(size, act, dtype):
    linear_backward_case(*size, dtype, act)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("xl", ["row", "pad", "off", "col"])
@pytest.mark.parametrize("wl", ["row", "off", "col", "colpad"])
def test_linear_backward_layouts(xl, wl, dtype):
    linear_backward_case(72, 136, 88, dtype, "silu", xl, wl)
    linear_backward_case(45, 71, 33, dtype, "none", xl, wl, dyl="pad")
    linear_backward_case(48, 72, 40, dtype, "none", xl, wl, dyl="col", bias=False)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_linear_backward_large(dtype):
    linear_backward_case(2048, 2048, 512, dtype, "gelu_tanh")
    linear_backward_case(300, 4096, 2560, dtype, "none")


def gated_case(m, n, k, dtype, act="silu", xl="row", wl="row", save=True, seed=0):
    d = Draw(seed * 65537 + m * 3 + n * 5 + k, dtype)
    x = d(m, k, xl)
    s = k ** -0.5 if k else 1.0
    wg, wu = d(n, k, wl, s), d(n, k, wl, s)
    r = llar.gated_ffn(x, wg, wu, activation=act, save=save)
    X = x.double()
    g, u = mm64(X, wg.double().t()), mm64(X, wu.double().t())
    ge = (k + 16) * EPS * mm64(X.abs(), wg.double().t().abs())
    ue = (k + 16) * EPS * mm64(X.abs(), wu.double().t().abs())
    h = r[0] if save else r
    v = act64(g, act)
    ve = 1.2 * ge + 16 * EPS * v.abs()
    if save:
        check(r[1], g, ge, "gate")
        check(r[2], u, ue, "up")
    check(h, v * u, ve * u.abs() + v.abs() * ue + ve * ue + EPS * (v * u).abs(), "gated %s" % ((m, n, k, dtype, act),))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gated_sizes(size, dtype):
    gated_case(*size, dtype)
    gated_case(*size, dtype, save=False, act="gelu", seed=1)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("wl", ["row", "off", "col", "colpad"])
def test_gated_activations_and_layouts(act, wl, dtype):
    gated_case(40, 72, 64, dtype, act, wl=wl)
    gated_case(5, 56, 264, dtype, act, wl=wl, xl="pad")
    gated_case(37, 45, 33, dtype, act, wl=wl, xl="col")


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("size", [(2048, 1152, 512), (4096, 2048, 128), (48, 3584, 1024), (513, 1032, 264)], ids=str)
def test_gated_large(size, dtype):
    gated_case(*size, dtype)
    gated_case(*size, dtype, wl="col", save=False)


def gated_backward_case(m, n, k, dtype, act="silu", xl="row", wl="row", hl="row", seed=0):
    d = Draw(seed * 40503 + m * 11 + n * 19 + k, dtype)
    x = d(m, k, xl)
    s = k ** -0.5 if k else 1.0
    wg, wu = d(n, k, wl, s), d(n, k, wl, s)
    dh, g, u = d(m, n, hl), d(m, n, hl), d(m, n)
    dx, dwg, dwu = llar.gated_ffn_backward(dh, x, wg, wu, g, u, activation=act)
    X, G, UP, H = x.double(), g.double(), u.double(), dh.double()
    v, sl = act64(G, act), slope64(G, act)
    dg, du = H * UP * sl, H * v
    r = U[dtype] * 1.01
    eg = 20 * EPS * (H * UP).abs() * (1 + G.abs()) + r * dg.abs() + TINY[dtype]
    eu = 20 * EPS * du.abs() + r * du.abs() + TINY[dtype]
    WG, WU = wg.double(), wu.double()
    A = mm64(dg.abs(), WG.abs()) + mm64(du.abs(), WU.abs())
    check(dx, mm64(dg, WG) + mm64(du, WU), mm64(eg, WG.abs()) + mm64(eu, WU.abs()) + (2 * n + 16) * EPS * A, "dx")
    for got, dz, e, what in ((dwg, dg, eg, "dw_gate"), (dwu, du, eu, "dw_up")):
        check(got, mm64(dz.t(), X), mm64(e.t(), X.abs()) + (m + 16) * EPS * mm64(dz.t().abs(), X.abs()), what)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", [(1, 64, 64), (7, 33, 50), (64, 128, 96), (130, 257, 264), (515, 72, 40)], ids=str)
def test_gated_backward(size, act, dtype):
    gated_backward_case(*size, dtype, act)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("xl", ["row", "pad", "off", "col"])
@pytest.mark.parametrize("wl", ["row", "off", "col", "colpad"])
def test_gated_backward_layouts(xl, wl, dtype):
    gated_backward_case(72, 136, 88, dtype, "silu", xl, wl)
    gated_backward_case(45, 71, 33, dtype, "gelu", xl, wl, hl="off")


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_gated_backward_large(dtype):
    gated_backward_case(2048, 1024, 512, dtype)
    gated_backward_case(300, 2048, 1280, dtype, "gelu_tanh")


# ---- what the gradients mean ------------------------------------------------------

def directional(f, point, direction, h):
    """Central difference of a binary64 function of a list of tensors."""
    return (f([p + h * d for p, d in zip(point, direction)]) - f([p - h * d for p, d in zip(point, direction)])) / (2 * h)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_match_differences(act):
    """binary32 gradients against central differences of the formula in binary64 (truncation h^2, rounding
    2^-53 / h: below 1e-8 here), along random directions; the gradients' own error is about sqrt(k) 2^-23."""
    d = Draw(77, torch.float32)
    m, n, k = 24, 40, 32
    x, wg, wu, c, b = d(m, k), d(n, k, scale=k ** -0.5), d(n, k, scale=k ** -0.5), d(m, n), d(1, n)[0]
    h, g, u = llar.gated_ffn(x, wg, wu, activation=act, save=True)
    grads = llar.gated_ffn_backward(c, x, wg, wu, g, u, activation=act)
    C = c.double()

    def gated(p):
        return (act64(p[0] @ p[1].t(), act) * (p[0] @ p[2].t()) * C).sum()

    def lin(p):
        return (act64(p[0] @ p[1].t() + p[2], act) * C).sum()

    y, z = llar.linear(x, wg, b, activation=act, save=True)
    lgrads = llar.linear_backward(c, x, wg, z, activation=act, bias_grad=True)
    for f, point, gr in ((gated, (x, wg, wu), grads), (lin, (x, wg, b), lgrads)):
        point = [p.double() for p in point]
        for i in range(3):
            direction = [torch.zeros_like(p) for p in point]
            direction[i] = d(*point[i].shape).double() if point[i].dim() == 2 else d(1, n)[0].double()
            # relu has kinks: a step that crosses one in z is off by that element's jump, so it is kept small
            step = 1e-5 if act != "relu" else 1e-9
            want = directional(f, point, direction, step)
            got = (gr[i].double() * direction[i]).sum()
            size = (gr[i].double() * direction[i]).abs().sum()
            assert abs(got - want) <= 1e-5 * size + 1e-6, (act, i, got.item(), want.item())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_matches_differences_of_the_kernel(act):
    """The forward kernel's own central difference: with outputs near 1, step 2^-6 and 2^-24 roundings of m n
    outputs, noise 2^-18 sqrt(m n) |c|, truncation about 2^-12 of a third derivative below 2."""
    d = Draw(78, torch.float32)
    m, n, k = 16, 24, 32
    x, wg, wu, c = d(m, k), d(n, k, scale=k ** -0.5), d(n, k, scale=k ** -0.5), d(m, n)
    dirn = d(m, k, scale=k ** -0.5)
    h = 2.0 ** -6
    f = lambda t: (llar.gated_ffn(t, wg, wu, activation=act).double() * c.double()).sum()  # noqa: E731
    want = (f(x + h * dirn) - f(x - h * dirn)) / (2 * h)
    _, g, u = llar.gated_ffn(x, wg, wu, activation=act, save=True)
    dx, _, _ = llar.gated_ffn_backward(c, x, wg, wu, g, u, activation=act)
    got = (dx.double() * dirn.double()).sum()
    size = (dx.double() * dirn.double()).abs().sum()
    assert abs(got - want) <= 2e-3 * size + 1e-3


# ---- edges --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_zero_sizes(dtype):
    e = lambda *s: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    assert llar.linear(e(0, 8), e(4, 8)).shape == (0, 4)
    assert llar.linear(e(3, 8), e(0, 8)).shape == (3, 0)
    b, r = torch.ones(4, dtype=dtype, device="cuda"), torch.full((3, 4), 2.0, dtype=dtype, device="cuda")
    assert (llar.linear(e(3, 0), e(4, 0), b, r) == 3).all()
    assert (llar.gated_ffn(e(3, 0), e(4, 0), e(4, 0)) == 0).all()
    assert llar.gated_ffn(e(0, 8), e(4, 8), e(4, 8)).shape == (0, 4)
    dx, dw, db = llar.linear_backward(e(0, 4), e(0, 8), e(4, 8), bias_grad=True)
    assert dx.shape == (0, 8) and (dw == 0).all() and (db == 0).all() and dw.shape == (4, 8)
    dx, dw, db = llar.linear_backward(e(3, 0), e(3, 8), e(0, 8), bias_grad=True)
    assert (dx == 0).all() and dx.shape == (3, 8) and dw.shape == (0, 8) and db.shape == (0,)
    dx, a, c = llar.gated_ffn_backward(e(0, 4), e(0, 8), e(4, 8), e(4, 8), e(0, 4), e(0, 4))
    assert dx.shape == (0, 8) and (a == 0).all() and (c == 0).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_leading_dimensions_vectors_and_broadcast_rows(dtype):
    d = Draw(5, dtype)
    x, w = d(6, 64), d(40, 64)
    y = llar.linear(x, w)
    assert torch.equal(llar.linear(x.view(2, 3, 64), w), y.view(2, 3, 40))
    assert torch.equal(llar.linear(x[1], w), llar.linear(x[1:2], w)[0])
    wide = x[2:3].expand(5, 64)
    assert torch.equal(llar.linear(wide, w), llar.linear(wide.contiguous(), w))
    r = d(1, 40)
    assert torch.equal(llar.linear(x, w, residual=r.expand(6, 40)), llar.linear(x, w, residual=r.repeat(6, 1)))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_infinities_and_nans_stay_where_they_belong(dtype):
    """An infinity makes its row's outputs infinite with the weight's sign (NaN against a zero weight), a NaN
    its row NaN, and no other row sees either."""
    for m, n, k in ((5, 48, 64), (80, 72, 136), (300, 264, 64)):
        d = Draw(9 + m, dtype)
        x, w = d(m, k), d(n, k)
        w[3, 2] = 0
        x[1, 2] = float("inf")
        x[2, 5] = float("-inf")
        x[4, 0] = float("nan")
        y = llar.linear(x, w)
        sign = torch.sign(w[:, 2].float())
        want = torch.where(sign == 0, torch.full_like(sign, float("nan")), sign * float("inf"))
        assert torch.equal(torch.nan_to_num(y[1].float(), nan=7.0), torch.nan_to_num(want, nan=7.0))
        assert torch.equal(y[2].float(), -torch.sign(w[:, 5].float()) * float("inf"))
        assert y[4].isnan().all()
        keep = [i for i in range(m) if i not in (1, 2, 4)]
        assert torch.equal(y[keep], llar.linear(torch.nan_to_num(x, 0, 0, 0), w)[keep])


def test_binary32_keeps_large_small_and_close_values():
    """Values at the ends of binary32's range, and a cancellation that needs all 24 bits."""
    x = torch.zeros(3, 64, device="cuda")
    w = torch.zeros(16, 64, device="cuda")
    x[0, 0], w[0, 0] = 3.4028234e38, 1.0      # rounds to infinity in bfloat16
    x[1, 1], w[1, 1] = 2.0 ** -100, 2.0 ** 20
    x[2, 2], x[2, 3], w[2, 2], w[2, 3] = 1 + 2.0 ** -23, -1.0, 1.0, 1.0
    y = llar.linear(x, w)
    assert y[0, 0].item() == torch.tensor(3.4028234e38).item()
    assert y[1, 1].item() == 2.0 ** -80
    assert y[2, 2].item() == 2.0 ** -23


@pytest.mark.parametrize("act", ACTS)
def test_activation_ends(act):
    """Far negative and far positive values: the activations' and slopes' limits, no NaN."""
    z = torch.tensor([[-float("inf"), -3e38, -1e4, -90.0, -0.0, 0.0, 90.0, 1e4, 3e38, float("inf")]], device="cuda")
    n = z.shape[1]
    y = llar.linear(torch.zeros(1, 1, device="cuda"), torch.zeros(n, 1, device="cuda"), z[0], activation=act)
    if act == "none":
        assert torch.equal(y, z)
    else:
        assert (y[0, :5].abs() < 1e-30).all() and torch.equal(y[0, 5:], z[0, 5:])
    dx, _, db = llar.linear_backward(torch.ones_like(z), torch.zeros(1, 1, device="cuda"),
                                     torch.zeros(n, 1, device="cuda"), z, activation=act, bias_grad=True)
    mid = {"none": 1.0, "relu": 0.0}.get(act, 0.5)
    low = 1.0 if act == "none" else 0.0
    want = torch.tensor([low] * 4 + [mid] * 2 + [1.0] * 4, device="cuda")
    assert torch.allclose(db, want, atol=1e-30, rtol=1e-6), db


def test_residual_may_be_the_output():
    for m, k in ((4, 2048), (70, 72), (64, 4096)):
        d = Draw(3, torch.bfloat16)
        x, w, r = d(m, k), d(136, k), d(m, 136)
        want = llar.linear(x, w, residual=r)
        got = llar.linear(x, w, residual=r, out=r)
        assert got is r and torch.equal(got, want)


def test_output_in_a_wider_buffer_leaves_its_surroundings():
    d = Draw(4, torch.bfloat16)
    for m, n, k in ((5, 72, 64), (130, 200, 72), (64, 77, 520)):
        x, w = d(m, k), d(n, k)
        buf = torch.full((m + 2, n + 5), 9.0, dtype=torch.bfloat16, device="cuda")
        llar.linear(x, w, out=buf[1:m + 1, 2:n + 2])
        assert torch.equal(buf[1:m + 1, 2:n + 2], llar.linear(x, w))
        buf[1:m + 1, 2:n + 2] = 9.0
        assert (buf == 9).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_same_bits_every_time(dtype):
    d = Draw(6, dtype)
    for m, n, k in ((1, 512, 4096), (64, 256, 4096), (300, 320, 520)):
        x, wg, wu, dh = d(m, k), d(n, k), d(n, k), d(m, n)
        a = llar.gated_ffn(x, wg, wu, save=True)
        g = llar.gated_ffn_backward(dh, x, wg, wu, a[1], a[2])
        y = llar.linear_backward(dh, x, wg, a[1], activation="gelu", bias_grad=True)
        for _ in range(3):
            for p, q in zip(a + g + y, llar.gated_ffn(x, wg, wu, save=True)
                            + llar.gated_ffn_backward(dh, x, wg, wu, a[1], a[2])
                            + llar.linear_backward(dh, x, wg, a[1], activation="gelu", bias_grad=True)):
                assert torch.equal(p, q)


def test_another_stream_and_a_graph():
    d = Draw(8, torch.bfloat16)
    x, wg, wu, wd = d(64, 1024), d(256, 1024), d(256, 1024), d(1024, 256)
    want = llar.linear(llar.gated_ffn(x, wg, wu), wd, residual=x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = llar.linear(llar.gated_ffn(x, wg, wu, stream=s), wd, residual=x, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = llar.linear(llar.gated_ffn(x, wg, wu), wd, residual=x)
    for i in range(3):
        x.copy_(d(64, 1024))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, llar.linear(llar.gated_ffn(x, wg, wu), wd, residual=x)), i


def test_refusals():
    d = Draw(1, torch.bfloat16)
    x, w = d(4, 64), d(32, 64)
    for bad in (lambda: llar.linear(x, w, activation="swish"),
                lambda: llar.linear(x, d(32, 48)),
                lambda: llar.linear(x, w.float()),
                lambda: llar.linear(x, w, bias=d(1, 31)[0]),
                lambda: llar.linear(x, w, bias=d(32, 2)[:, 0]),
                lambda: llar.linear(x, w, residual=d(4, 31)),
                lambda: llar.linear(x, w, out=d(5, 32)),
                lambda: llar.linear(x.cpu(), w),
                lambda: llar.linear(d(4, 128)[:, ::2], w),            # no axis of stride 1
                lambda: llar.linear(x, w, out=d(32, 4).t()),          # output columns not contiguous
                lambda: llar.linear(x, w, residual=d(32, 4).t()),
                lambda: llar.linear(d(2, 3, "row").new_empty(2, 3, 64).transpose(0, 1), w),
                lambda: llar.gated_ffn(x, w, d(32, 64, "pad")),       # other strides
                lambda: llar.gated_ffn(x, w, d(31, 64)),
                lambda: llar.gated_ffn_backward(d(4, 32), x, w, w, d(4, 32), d(4, 30)),
                lambda: llar.linear_backward(d(4, 32), x, w, activation="silu"),
                lambda: llar.linear_backward(d(4, 31), x, w)):
        with pytest.raises((ValueError, TypeError, llar.LlarError)):
            bad()
    with pytest.raises(TypeError):
        llar.linear(x.double(), w.double())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=ids)
@pytest.mark.parametrize("k", [500, 512, 576, 640, 1160])
def test_residual_of_large_tiles(k, dtype):
    """The residual taken while the sums grow (nine k tiles or more) and before them (fewer); rows and columns
    that end inside a tile; residuals whose rows are apart, unaligned, repeated, or the output itself."""
    m, n = 3000, 4104
    d = Draw(k, dtype)
    w, b = d(n, k, "row", k ** -0.5), d(1, n)[0]
    for xl in ("row", "col"):
        x = d(m, k, xl)
        X, W = x.double(), w.double()
        want, A = mm64(X, W.t()), mm64(X.abs(), W.t().abs())
        for rl in ("row", "pad", "off", "one", "out"):
            r = d(1, n).expand(m, n) if rl == "one" else d(m, n, "row" if rl == "out" else rl)
            bias = b if rl in ("row", "off") else None
            w64, a64 = want + r.double(), A + r.double().abs()
            if bias is not None:
                w64, a64 = w64 + b.double(), a64 + b.double().abs()
            y = llar.linear(x, w, bias, r, out=r if rl == "out" else None)
            check(y, w64, (k + 16) * EPS * a64, "residual %s, x %s" % (rl, xl))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("size", [(48, 2560, 1280), (90, 64, 1500), (2400, 320, 290), (515, 500, 1410), (1030, 2048, 520)],
                         ids=str)
def test_both_gradients_of_one_launch(size, dtype):
    """They are what each of them is alone, up to the order of the sums; and the same bits every time."""
    m, n, k = size
    d = Draw(m, dtype)
    x, w, dy = d(m, k), d(n, k, "row", k ** -0.5), d(m, n)
    dx, dw, _ = llar.linear_backward(dy, x, w)
    X, W, Y = x.double(), w.double(), dy.double()
    check(dx, mm64(Y, W), (n + 16) * EPS * mm64(Y.abs(), W.abs()), "dx")
    check(dw, mm64(Y.t(), X), (m + 16) * EPS * mm64(Y.t().abs(), X.abs()), "dw")
    for _ in range(3):
        again = llar.linear_backward(dy, x, w)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    only_dx = llar.linear_backward(dy, x, w, weight_grad=False)
    only_dw = llar.linear_backward(dy, x, w, input_grad=False)
    assert only_dx[1] is None and only_dw[0] is None
    check(only_dx[0], mm64(Y, W), (n + 16) * EPS * mm64(Y.abs(), W.abs()), "dx alone")
    check(only_dw[1], mm64(Y.t(), X), (m + 16) * EPS * mm64(Y.t().abs(), X.abs()), "dw alone")


def test_lines_far_apart():
    """Rows 8 MiB and more apart (copied above 16 rows, read in place below), offsets beyond 2^32 elements, and an
    output and a residual whose rows are as far apart."""
    dtype, n, k, ld = torch.bfloat16, 40, 72, (1 << 27) + 8
    big = torch.empty(n * ld, dtype=dtype, device="cuda")

    def far(rows, cols, start):
        return big[start:].as_strided((rows, cols), (ld, 1))
    w = far(n, k, 0)
    d = Draw(5, dtype)
    w.copy_(d(n, k))
    assert (n - 1) * ld > 1 << 32
    for m in (1, 4, 40):
        x = d(m, k)
        assert torch.equal(llar.linear(x, w), llar.linear(x, w.contiguous()))
        xf, rf, out = far(m, k, 1024), far(m, n, 2048), far(m, n, 4096)
        xf.copy_(x)
        rf.copy_(d(m, n))
        want = llar.linear(x, w.contiguous(), residual=rf.contiguous())
        assert llar.linear(xf, w, residual=rf, out=out) is out
        assert torch.equal(out, want)
        dy = far(m, n, 8192)
        dy.copy_(d(m, n))
        for a, b in zip(llar.linear_backward(dy, xf, w, bias_grad=True),
                        llar.linear_backward(dy.contiguous(), x, w.contiguous(), bias_grad=True)):
            assert torch.equal(a, b)
