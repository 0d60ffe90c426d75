"""What binary32 products keep of their operands' 24 bits.

An operand is three bfloat16 parts: hi, mid (at most 2^-8 of the value's power
of two) and lo (at most 2^-17).  The products of parts left out, mid lo twice
and lo lo, are at most 2^-24 (1 + 2^-10) of the whole.  The six kept ones are
exact and added smallest first: where one product is all there is, the first
five sums stay below 2^-6 of it and round by at most 2^-23 of that each, and the
last by at most 2^-23.  Altogether below 1.6 x 2^-23 of the product."""
import pytest
import torch

import message_allreduce_amd as llar

pytestmark = pytest.mark.gpu

TOL = 1.6 * 2.0 ** -23
# few rows; then products that want each tile shape, whole in k and split between workgroups
SIZES = [(1, 40, 72), (3, 72, 96), (16, 520, 1000), (17, 40, 200), (17, 40, 4000), (40, 136, 72), (200, 2000, 1000),
         (300, 264, 136), (500, 4100, 40), (2000, 2000, 200), (3000, 1000, 2000)]


def numbers(rows, cols, seed):
    """Normal values, every third with the mantissa whose parts are the largest when cut or rounded."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.empty(rows, cols, device="cuda").normal_(generator=g)
    bits = t.view(torch.int32).flatten()
    bits[::6] = (bits[::6] & -8388608) | 0x0000ffff
    bits[3::6] = (bits[3::6] & -8388608) | 0x00007f7f
    return t


def one_each(rows, cols, values):
    """values[i] alone in row i; the row's place, and the matrix."""
    at = (torch.arange(rows, device="cuda") * 7 + 3) % cols
    m = torch.zeros(rows, cols, device="cuda")
    m[torch.arange(rows, device="cuda"), at] = values
    return m, at


def ordered(t, layout):
    return t if layout == "row" else t.t().contiguous().t()


def close(got, want, what):
    off = (got.double() - want).abs()
    assert (off <= TOL * want.abs()).all(), "%s: off by %.3g x 2^-23" % (what, (off / want.abs()).max() * 2 ** 23)


@pytest.mark.parametrize("xl", ["row", "col"])
@pytest.mark.parametrize("wl", ["row", "col"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_single_products(size, wl, xl):
    m, n, k = size
    v, w, wu = numbers(m, 1, m)[:, 0], numbers(n, k, n + k), numbers(n, k, n * k)
    x, at = one_each(m, k, v)
    x, wo, wuo = ordered(x, xl), ordered(w, wl), ordered(wu, wl)
    want, up = (v.double()[:, None] * t.double().t()[at] for t in (w, wu))
    close(llar.linear(x, wo), want, "linear")
    _, g, u = llar.gated_ffn(x, wo, wuo, activation="none", save=True)
    close(g, want, "gate")
    close(u, up, "up")


@pytest.mark.parametrize("wl", ["row", "col"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_single_products_of_gradients(size, wl):
    m, n, k = size
    # dx: one output's gradient a token
    v, w = numbers(m, 1, m)[:, 0], numbers(n, k, n + k)
    dy, at = one_each(m, n, v)
    x = numbers(m, k, k)
    dx, _, _ = llar.linear_backward(dy, x, ordered(w, wl))
    close(dx, v.double()[:, None] * w.double()[at], "dx")
    # dw: one token's gradient an output
    v = numbers(n, 1, n)[:, 0]
    dyt, at = one_each(n, m, v)
    want = v.double()[:, None] * x.double()[at]
    _, dw, _ = llar.linear_backward(dyt.t().contiguous(), x, ordered(w, wl))
    close(dw, want, "dw")
    _, dw, _ = llar.linear_backward(dyt.t().contiguous(), x, ordered(w, wl), input_grad=False)
    close(dw, want, "dw alone")
    one = torch.ones(m, n, device="cuda")
    _, dwg, dwu = llar.gated_ffn_backward(dyt.t().contiguous(), x, ordered(w, wl), ordered(w, wl), one, one,
                                          activation="none")
    close(dwg, want, "dw_gate")
    close(dwu, want, "dw_up")


@pytest.mark.parametrize("wl", ["row", "col"])
@pytest.mark.parametrize("m", [3, 16, 40, 300])
def test_values_at_the_ends_of_the_range_and_cancellation(m, wl):
    big = torch.finfo(torch.float32).max
    k, n = 72, 264
    x = torch.zeros(m, k, device="cuda")
    w = torch.zeros(n, k, device="cuda")
    x[0, 0], w[0, 0] = big, 1.0                    # rounds to infinity in bfloat16
    x[1, 1], w[1, 1] = -big, 0.5
    x[1, 0] = 1.0
    x[2, 2], x[2, 70], w[2, 2], w[2, 70] = 1 + 2.0 ** -23, -1.0, 1.0, 1.0
    x[2, 3], w[3, 3] = 2.0 ** -100, 2.0 ** 20
    x[0, 5] = w[5, 5] = 2.0 ** 64 * (1 - 2.0 ** -10)  # the first parts' product overflows, the whole does not
    x[0, 71], w[6, 71] = big, 2.0                     # overflows
    y = llar.linear(x, ordered(w, wl))
    assert y[0, 0].item() == big and y[0, 6].item() == float("inf")
    assert y[0, 5].item() == float((x[0, 5] * w[5, 5]).item())
    assert (y[0, 1:5] == 0).all() and (y[0, 7:] == 0).all()
    assert y[1, 1].item() == -big / 2 and y[1, 0].item() == 1.0 and (y[1, 2:] == 0).all()
    assert y[2, 2].item() == 2.0 ** -23 and y[2, 3].item() == 2.0 ** -80
    assert (y[3:] == 0).all()


@pytest.mark.parametrize("m", [3, 16, 40, 300])
def test_small_values_keep_what_the_parts_can_hold(m):
    """A bfloat16 has no bits below 2^-133: that much of a value's third part may be lost."""
    scale = 2.0 ** (-140 + torch.arange(m, device="cuda").double() * 11 % 40)
    v = (numbers(m, 1, m)[:, 0].double() * scale).float()
    x, at = one_each(m, 72, v)
    w = torch.full((264, 72), 2.0 ** 40, device="cuda")
    want = v.double()[:, None] * 2.0 ** 40
    off = (llar.linear(x, w).double() - want).abs()
    assert (off <= TOL * want.abs() + 2.0 ** (40 - 133)).all()


def same_kind(got, want, what):
    """Infinities, with their signs, and NaNs are where binary64 has them; the rest is near."""
    assert torch.equal(got.isnan(), want.isnan()), what
    assert torch.equal(got == float("inf"), want == float("inf")), what
    assert torch.equal(got == -float("inf"), want == -float("inf")), what
    ok = want.isfinite()
    assert torch.allclose(got[ok].double(), want[ok], rtol=1e-4, atol=1e-4), what


@pytest.mark.parametrize("wl", ["row", "col"])
@pytest.mark.parametrize("size", [(5, 48, 64), (16, 72, 1000), (40, 56, 72), (17, 40, 4000), (300, 264, 136)], ids=str)
def test_infinities_go_through_both_products_and_splits(size, wl):
    """An infinity, two of opposite weight, and a NaN, in either of the pairs that are added, in the first, a
    middle and the last k: the sums taken again run over the same products."""
    m, n, k = size
    g = torch.Generator(device="cuda")
    g.manual_seed(m * n)
    def t(r, c):
        return torch.empty(r, c, device="cuda").normal_(generator=g)
    inf, nan = float("inf"), float("nan")
    wg, wu, x = t(n, k), t(n, k), t(m, k)
    wgo, wuo = ordered(wg, wl), ordered(wu, wl)
    xi = x.clone()
    xi[0, k - 1], xi[1, k // 2], xi[2, 0], xi[2, k - 1], xi[3, k // 2] = inf, -inf, inf, inf, nan
    for got, w in zip(llar.gated_ffn(xi, wgo, wuo, activation="none", save=True)[1:], (wg, wu)):
        same_kind(got, torch.mm(xi.double(), w.double().t()), "forward")
    same_kind(llar.linear(xi, wgo), torch.mm(xi.double(), wg.double().t()), "linear")
    one = torch.ones(m, n, device="cuda")
    for pair in (0, 1):
        for at in (0, n // 2, n - 1):
            # activation none: dg = dh up, du = dh gate
            gate, up = one.clone(), one.clone()
            (up if pair == 0 else gate)[1, at] = inf
            (up if pair == 0 else gate)[2, at] = nan
            dh = t(m, n)
            dx, dwg, dwu = llar.gated_ffn_backward(dh, x, wgo, wuo, gate, up, activation="none")
            dg, du = dh.double() * up.double(), dh.double() * gate.double()
            same_kind(dx, torch.mm(dg, wg.double()) + torch.mm(du, wu.double()), "dx")
            same_kind(dwg, torch.mm(dg.t().contiguous(), x.double()), "dw_gate")
            same_kind(dwu, torch.mm(du.t().contiguous(), x.double()), "dw_up")
