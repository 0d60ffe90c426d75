"""The 8-bit products and the quantisation before them against their definitions in binary64.

Tolerances.  Quantisation is exact: q and scale are what binary64 gives.  A whole
sum (exact) becomes a value by three roundings of binary32 (to binary32, times
each scale): 3 x 2^-24 of it, and 2^-149 for each where it is tiny.  The bias adds
one; an activation of slope at most 1.2 passes that on and is itself evaluated to
16 roundings of binary32; the output rounds once (test_gpu_ffn.check).
"""
import math

import pytest
import torch

import message_allreduce_amd as llar
from test_gpu_ffn import ACTS, DTYPES, EPS, Draw, act64, check, ids, mm64

pytestmark = pytest.mark.gpu


def quantized64(x):
    """The definition, in binary64 but for scale's rounding."""
    x = x.double()
    top = x.abs().amax(1) if x.shape[1] else x.new_zeros(x.shape[0])
    scale = (top / 127).float()
    s = scale.double()[:, None]
    q = torch.round(x / torch.where(s > 0, s, torch.ones_like(s))).clamp(-127, 127)
    fine = torch.isfinite(s) & (s > 0)
    q = torch.where(fine, q, torch.zeros_like(q))
    return q, torch.where(torch.isfinite(scale), scale, torch.full_like(scale, math.nan))


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=-7.0), torch.nan_to_num(b, nan=-7.0))


def quantize_case(x):
    q, scale = llar.quantize_rows(x)
    assert q.dtype == torch.int8 and scale.dtype == torch.float32 and q.shape == x.shape and scale.shape == x.shape[:-1]
    wq, ws = quantized64(x.reshape(-1, x.shape[-1]))
    assert same(scale.reshape(-1), ws), (scale.reshape(-1) - ws).abs().max()
    bad = q.reshape(wq.shape).double() != wq
    assert not bad.any(), (bad.nonzero()[0].tolist(), int(bad.sum()))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("layout", ["row", "pad", "off", "col", "colpad"])
def test_quantize_sizes_and_layouts(layout, dtype):
    for rows, k in ((1, 1), (1, 8), (3, 7), (5, 130), (9, 2048), (4, 2049), (2, 8192), (3, 8200), (70, 520), (2, 20001),
                    (64, 33), (200, 1), (129, 2047), (1100, 40), (1030, 2500), (1024, 9000)):
        quantize_case(Draw(rows + k, dtype)(rows, k, layout))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_quantize_ties_and_ends(dtype):
    """Exact halves, on both sides and next to them; rows of zeros, tiny and huge ones, infinities and NaN."""
    x = torch.zeros(12, 300, device="cuda", dtype=torch.float64)
    half = torch.arange(-127, 128, dtype=torch.float64, device="cuda") - 0.5
    x[0, 0], x[0, 1:256] = 127.0, half                        # scale 1: every half but -127.5
    x[1] = x[0] * 2.0 ** -100
    x[2, 0], x[2, 1:256] = 254.0, 2 * half
    x[3, 5] = 1e-7                                            # one value
    x[4] = torch.linspace(-1, 1, 300, device="cuda") * torch.finfo(dtype).max
    x[5] = torch.linspace(-1, 1, 300, device="cuda") * torch.finfo(dtype).tiny
    x[6] = torch.arange(300, device="cuda") * torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps  # subnormal
    x[7, 9], x[7, 10] = math.inf, 1.0
    x[8, 0], x[8, 299] = -math.inf, math.nan
    x[9, 150] = math.nan
    x[10, 0] = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps  # the least magnitude
    x = x.to(dtype)
    x[0, 0] = 127.0
    near = x[0].float()
    near = torch.nextafter(near, near * 2).to(dtype)          # binary32: just beyond each half
    quantize_case(torch.cat([x, near[None], -near[None]]))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_quantize_shapes(dtype):
    d = Draw(3, dtype)
    x = d(6, 40)
    q, s = llar.quantize_rows(x)
    q3, s3 = llar.quantize_rows(x.view(2, 3, 40))
    assert q3.shape == (2, 3, 40) and s3.shape == (2, 3) and torch.equal(q3.view(6, 40), q) and torch.equal(s3.view(6), s)
    q1, s1 = llar.quantize_rows(x[2])
    assert q1.shape == (40,) and s1.shape == () and torch.equal(q1, q[2]) and s1 == s[2]
    assert torch.equal(llar.quantize_rows(x[1:2].expand(4, 40))[0], q[1:2].expand(4, 40))
    for shape in ((0, 40), (3, 0), (0, 0)):
        q, s = llar.quantize_rows(torch.empty(shape, dtype=dtype, device="cuda"))
        assert q.shape == shape and s.shape == shape[:1] and (s == 0).all()


class Draw8:
    """Whole numbers of the whole range, -128 among them, in matrices as test_gpu_ffn.Draw lays them out."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def __call__(self, rows, cols, layout="row"):
        wide = {"row": 0, "pad": 16, "off": 3}[layout]
        t = torch.randint(-128, 128, (rows, cols + wide), dtype=torch.int8, device="cuda", generator=self.g)
        return t[:, 1:cols + 1] if layout == "off" else t[:, :cols]

    def scales(self, n, k=1):
        return torch.empty(n, device="cuda").uniform_(0.5, 2.0, generator=self.g) / (74 * max(k, 1) ** 0.5)


def value64(q, qs, w, ws):
    """The products' values and what the kernel's may be off."""
    z = mm64(q.double(), w.double().t()) * qs.double()[:, None] * ws.double()
    return z, 3.03 * 2.0 ** -24 * z.abs() + 3 * 2.0 ** -149


def linear_case(m, n, k, dtype, act="none", bias=False, residual=False, given=True, xl="row", wl="row", seed=0, out=None):
    d, d8 = Draw(seed + m * 31 + n, dtype), Draw8(seed * 7919 + m * 31 + n * 17 + k)
    w, ws = d8(n, k, wl), d8.scales(n, k)
    b = d(1, n)[0] if bias else None
    r = d(m, n) if residual else None
    if given:
        x, xs = d8(m, k, xl), d8.scales(m)
        q, qs = x, xs
    else:
        x, xs = d(m, k, xl), None
        q, qs = quantized64(x)
    y = llar.linear_int8(x, w, ws, x_scale=xs, bias=b, residual=r, activation=act, dtype=dtype if given else None, out=out)
    assert y.dtype == dtype
    z, err = value64(q, qs, w, ws)
    if bias:
        z = z + b.double()
        err = err + 2.0 ** -24 * 1.01 * z.abs()
    want = act64(z, act)
    if act != "none":
        err = 1.2 * err + 16 * EPS * want.abs()
    if residual:
        want, err = want + r.double(), err + EPS * (want.abs() + r.double().abs())
    check(y, want, err, "linear_int8 %s" % ((m, n, k, dtype, act, given, xl, wl),))
    return y


# rows on both sides of 8, 16 and 32, and products that want each tile shape, whole in k and split between workgroups
SIZES = [(1, 1, 1), (1, 512, 512), (1, 77, 130), (2, 64, 8), (2, 40, 5000), (3, 200, 96), (16, 64, 64), (16, 33, 8200),
         (17, 33, 65), (31, 129, 72), (64, 64, 2048), (65, 640, 320), (128, 128, 128), (200, 513, 257), (257, 256, 64),
         (300, 264, 1000), (64, 40, 20000)]
LARGE = [(9, 16500, 80), (16, 16600, 300), (20, 72, 8000), (31, 8200, 200), (32, 8100, 200), (17, 4100, 4000),
         (40, 72, 128), (100, 1096, 2000), (200, 2000, 8000), (500, 4100, 80), (500, 4104, 400),
         (1000, 2000, 1008), (2000, 2000, 400), (2000, 4100, 80), (3000, 40, 4000), (3000, 4104, 1280), (4096, 4096, 256)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_linear_sizes(size, dtype):
    linear_case(*size, dtype)
    linear_case(*size, dtype, given=False)
    linear_case(*size, dtype, "gelu", True, True, seed=1)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("size", LARGE, ids=str)
def test_linear_large(size, dtype):
    linear_case(*size, dtype)
    linear_case(*size, dtype, "silu", True, True, given=False)
    linear_case(*size, dtype, "none", False, True)
    linear_case(*size, dtype, "none", True, False)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("xl", ["row", "pad", "off"])
@pytest.mark.parametrize("wl", ["row", "pad", "off"])
def test_linear_layouts(xl, wl, dtype):
    for size in ((72, 136, 96), (33, 71, 45), (1, 40, 64), (9, 264, 520), (2, 71, 45)):
        linear_case(*size, dtype, bias=True, xl=xl, wl=wl)
        linear_case(*size, dtype, given=False, xl=xl, wl=wl)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("xl", ["col", "colpad"])
def test_linear_quantizes_any_layout(xl, dtype):
    for size in ((72, 136, 96), (33, 71, 45), (9, 264, 520), (2, 40, 64)):
        linear_case(*size, dtype, given=False, xl=xl)
    d, d8 = Draw(1, dtype), Draw8(2)
    w, ws = d8(40, 32), d8.scales(40, 32)
    for m in (2, 40):
        x = d(m, 64)[:, ::2]  # neither axis contiguous
        assert torch.equal(llar.linear_int8(x, w, ws), llar.linear_int8(x.contiguous(), w, ws))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("act", ACTS)
def test_linear_epilogues(act, dtype):
    for bias in (False, True):
        for residual in (False, True):
            for size in ((40, 72, 64), (1, 72, 1024), (4, 72, 1024), (48, 72, 8192)):
                linear_case(*size, dtype, act, bias, residual)


def gated_case(m, n, k, dtype, act="silu", given=True, xl="row", wl="row", seed=0):
    d, d8 = Draw(seed + m, dtype), Draw8(seed * 65537 + m * 3 + n * 5 + k)
    wg, wu, gs, us = d8(n, k, wl), d8(n, k, wl), d8.scales(n, k), d8.scales(n, k)
    if given:
        x, xs = d8(m, k, xl), d8.scales(m)
        q, qs = x, xs
    else:
        x, xs = d(m, k, xl), None
        q, qs = quantized64(x)
    h = llar.gated_ffn_int8(x, wg, wu, gs, us, x_scale=xs, activation=act, dtype=dtype)
    g, ge = value64(q, qs, wg, gs)
    u, ue = value64(q, qs, wu, us)
    v = act64(g, act)
    ve = 1.2 * ge + 16 * EPS * v.abs()
    check(h, v * u, ve * u.abs() + v.abs() * ue + ve * ue + EPS * (v * u).abs(), "gated_int8 %s" % ((m, n, k, act, given),))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("size", SIZES + LARGE, ids=str)
def test_gated_sizes(size, dtype):
    gated_case(*size, dtype)
    gated_case(*size, dtype, "gelu", given=False, seed=1)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("wl", ["row", "pad", "off"])
def test_gated_activations_and_layouts(act, wl, dtype):
    for size in ((40, 72, 64), (5, 56, 264), (37, 45, 33), (1, 45, 130)):
        gated_case(*size, dtype, act, wl=wl)
        gated_case(*size, dtype, act, given=False, wl=wl, xl="pad")


# ---- edges ---------------------------------------------------------------------------

@pytest.mark.parametrize("m", [1, 2, 5, 40, 300])
def test_sums_at_the_end_of_32_bits(m):
    """The longest k with the largest products: no partial or joined sum overflows."""
    k, n = (1 << 17) - 1, 24
    x = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    w[1], w[2, ::2] = 127, 127
    x[m - 1] = 127
    one, ws = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    y = llar.linear_int8(x, w, ws, x_scale=one, dtype=torch.float32)
    want = mm64(x.double(), w.double().t())
    assert want.abs().max() == 131071 * 16384 or m == 1
    assert torch.equal(y, want.float())


def test_scales_do_not_overflow_on_the_way():
    """A large sum times a small scale times a large one, and the other way round."""
    for m in (1, 3, 40):
        x = torch.full((m, 512), 127, dtype=torch.int8, device="cuda")
        w = torch.full((24, 512), 127, dtype=torch.int8, device="cuda")
        for a, b in ((1e-30, 1e25), (1e25, 1e-30), (1e-20, 1e-15), (2e36, 1e-7), (1e-38, 1e3)):
            xs, ws = torch.full((m,), a, device="cuda"), torch.full((24,), b, device="cuda")
            y = llar.linear_int8(x, w, ws, x_scale=xs, dtype=torch.float32).double()
            want = 512 * 127 * 127 * xs[0].double() * ws[0].double()
            assert ((y - want).abs() <= 3.03 * 2.0 ** -24 * want).all(), (m, a, b)


@pytest.mark.parametrize("m", [1, 4, 40])
def test_tokens_at_the_ends_of_the_range(m):
    """Values up to bfloat16's largest and down to its least, in one batch: no infinity and no zero on the way."""
    d8 = Draw8(m)
    x = Draw(m, torch.bfloat16)(m, 512)
    x = x / x.abs().amax(1, keepdim=True)
    x[m - 1] *= 3e38
    if m > 1:
        x[0] *= 1e-36
    w, ws = d8(24, 512), d8.scales(24, 512) * 1e-4
    y = llar.linear_int8(x, w, ws)
    q, qs = quantized64(x)
    want, err = value64(q, qs, w, ws)
    assert torch.isfinite(want.float()).all()
    check(y, want, err, "ends")


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_rows_that_are_not_finite_stay_apart(dtype):
    for m, n, k in ((5, 48, 64), (80, 72, 136), (300, 264, 64)):
        d, d8 = Draw(9 + m, dtype), Draw8(m)
        x, w, ws = d(m, k), d8(n, k), d8.scales(n, k)
        x[1, 2], x[2, 5], x[4, 0], x[3] = math.inf, -math.inf, math.nan, 0
        for y, clean in ((llar.linear_int8(x, w, ws), llar.linear_int8(torch.nan_to_num(x, 0, 0, 0), w, ws)),
                         (llar.gated_ffn_int8(x, w, w, ws, ws), llar.gated_ffn_int8(torch.nan_to_num(x, 0, 0, 0), w, w, ws, ws))):
            assert y[[1, 2, 4]].isnan().all() and (y[3] == 0).all()
            keep = [i for i in range(m) if i not in (1, 2, 4)]
            assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_zero_sizes(dtype):
    i8 = lambda *s: torch.empty(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    v = lambda *s: torch.ones(*s, dtype=dtype, device="cuda")  # noqa: E731
    assert llar.linear_int8(i8(0, 8), i8(4, 8), f(4), x_scale=f(0), dtype=dtype).shape == (0, 4)
    assert llar.linear_int8(v(0, 8), i8(4, 8), f(4)).shape == (0, 4)
    assert llar.linear_int8(v(3, 8), i8(0, 8), f(0)).shape == (3, 0)
    for m in (3, 40):
        assert (llar.linear_int8(v(m, 0), i8(4, 0), f(4), bias=v(4), residual=v(m, 4)) == 2).all()
        assert (llar.gated_ffn_int8(i8(m, 0), i8(4, 0), i8(4, 0), f(4), f(4), x_scale=f(m), dtype=dtype) == 0).all()
    assert llar.gated_ffn_int8(v(0, 8), i8(4, 8), i8(4, 8), f(4), f(4)).shape == (0, 4)


@pytest.mark.parametrize("m", [1, 2, 6, 60])
def test_shapes_outputs_and_residuals(m):
    """Leading dimensions, an output in a wider buffer, the residual as the output, bf16 by default."""
    d, d8 = Draw(m, torch.bfloat16), Draw8(m)
    x, xs, w, ws, r = d8(m, 64), d8.scales(m), d8(40, 64), d8.scales(40, 64), d(m, 40)
    y = llar.linear_int8(x, w, ws, x_scale=xs, residual=r)
    assert y.dtype == torch.bfloat16
    if m % 2 == 0:
        y3 = llar.linear_int8(x.view(2, -1, 64), w, ws, x_scale=xs.view(2, -1), residual=r.view(2, -1, 40))
        assert torch.equal(y3.view(m, 40), y)
    if m == 1:
        assert torch.equal(llar.linear_int8(x[0], w, ws, x_scale=xs[0], residual=r[0]), y[0])
    buf = torch.full((m + 2, 45), 9.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(llar.linear_int8(x, w, ws, x_scale=xs, residual=r, out=buf[1:m + 1, 2:42]), y)
    buf[1:m + 1, 2:42] = 9.0
    assert (buf == 9).all()
    rr = d(1, 40)
    assert torch.equal(llar.linear_int8(x, w, ws, x_scale=xs, residual=rr.expand(m, 40)),
                       llar.linear_int8(x, w, ws, x_scale=xs, residual=rr.repeat(m, 1)))
    assert llar.linear_int8(x, w, ws, x_scale=xs, residual=r, out=r) is r and torch.equal(r, y)


@pytest.mark.parametrize("m", [1, 2, 7, 64, 300])
def test_whole_numbers_given_or_made_are_the_same(m):
    """The call's own quantisation is quantize_rows', whichever kernel does it; and every call gives the same bits."""
    for dtype in DTYPES:
        d, d8 = Draw(m, dtype), Draw8(m)
        x, w, ws = d(m, 2500), d8(264, 2500), d8.scales(264, 2500)
        q, s = llar.quantize_rows(x)
        want = llar.linear_int8(q, w, ws, x_scale=s, dtype=dtype)
        wg = llar.gated_ffn_int8(q, w, w, ws, ws, x_scale=s, dtype=dtype)
        for _ in range(3):
            assert torch.equal(llar.linear_int8(x, w, ws), want)
            assert torch.equal(llar.gated_ffn_int8(x, w, w, ws, ws), wg)


def test_another_stream_and_a_graph():
    """A block of both products, with its own quantisations, on another stream and replayed."""
    for m in (1, 2, 12, 64):
        d, d8 = Draw(8, torch.bfloat16), Draw8(8)
        x = d(m, 1024)
        w = [(d8(256, 1024), d8.scales(256, 1024)), (d8(256, 1024), d8.scales(256, 1024)), (d8(1024, 256), d8.scales(1024, 256))]

        def block(stream=None):
            h = llar.gated_ffn_int8(x, w[0][0], w[1][0], w[0][1], w[1][1], stream=stream)
            q, s = llar.quantize_rows(h, stream=stream)
            y = llar.linear_int8(q, w[2][0], w[2][1], x_scale=s, residual=x, stream=stream)
            return y, llar.linear_int8(h, w[2][0], w[2][1], residual=x, stream=stream)

        want = block()
        assert torch.equal(want[0], want[1])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = block(s)
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = block()
        for i in range(3):
            x.copy_(d(m, 1024))
            graph.replay()
            torch.cuda.synchronize()
            now = block()
            assert torch.equal(out[0], now[0]) and torch.equal(out[1], now[1]), (m, i)


def test_lines_far_apart():
    """Rows 8 MiB and more apart (copied above 16 rows, read in place below), offsets beyond 2^32 elements."""
    n, k, ld = 40, 80, (1 << 27) + 16
    big = torch.empty(n * ld, dtype=torch.int8, device="cuda")

    def far(rows, cols, start):
        return big[start:].as_strided((rows, cols), (ld, 1))
    d8 = Draw8(5)
    w, ws = far(n, k, 0), d8.scales(n, k)
    w.copy_(d8(n, k))
    assert (n - 1) * ld > 1 << 32
    for m in (1, 2, 4, 40):
        x, xs = far(m, k, 1024), d8.scales(m)
        x.copy_(d8(m, k))
        want = llar.linear_int8(x.contiguous(), w.contiguous(), ws, x_scale=xs)
        assert torch.equal(llar.linear_int8(x, w, ws, x_scale=xs), want)


def test_wide_outputs_of_few_tokens():
    """More outputs than one launch of a workgroup per 16 of them takes."""
    n, k = (1 << 24) + 40, 16
    d8 = Draw8(1)
    w, ws, x, xs = d8(n, k), d8.scales(n, k), d8(2, k), d8.scales(2)
    y = llar.linear_int8(x, w, ws, x_scale=xs, dtype=torch.float32)
    for part in (slice(0, 4096), slice((1 << 24) - 2000, n)):
        z, err = value64(x, xs, w[part], ws[part])
        assert ((y[:, part].double() - z).abs() <= err).all()


def test_refusals():
    d, d8 = Draw(1, torch.bfloat16), Draw8(1)
    v, x, xs, w, ws = d(4, 64), d8(4, 64), d8.scales(4), d8(32, 64), d8.scales(32)
    lin, gat = llar.linear_int8, llar.gated_ffn_int8
    for bad in (lambda: lin(x, w, ws),                                     # int8 without scales
                lambda: lin(v, w, ws, x_scale=xs),                         # values with them
                lambda: lin(x, w, ws, x_scale=xs, dtype=torch.float64),
                lambda: lin(v, w, ws, dtype=torch.float16),
                lambda: lin(x, w, ws, x_scale=xs, activation="swish"),
                lambda: lin(x, w.float(), ws, x_scale=xs),
                lambda: lin(x, d8(32, 48), ws, x_scale=xs),
                lambda: lin(x, w, ws[:31], x_scale=xs),
                lambda: lin(x, w, ws.double(), x_scale=xs),
                lambda: lin(x, w, d8.scales(64)[::2], x_scale=xs),
                lambda: lin(x, w, ws, x_scale=xs[:3]),
                lambda: lin(x, w, ws, x_scale=xs.view(4, 1)),
                lambda: lin(x, w, ws, x_scale=d8.scales(8)[::2]),
                lambda: lin(x, w, ws.cpu(), x_scale=xs),
                lambda: lin(x, w, ws, x_scale=xs, bias=d(1, 31)[0]),
                lambda: lin(x, w, ws, x_scale=xs, bias=d(1, 32)[0].float()),
                lambda: lin(x, w, ws, x_scale=xs, residual=d(4, 32).float()),
                lambda: lin(x, w, ws, x_scale=xs, out=d(5, 32)),
                lambda: lin(x.cpu(), w, ws, x_scale=xs),
                lambda: lin(d8(4, 128)[:, ::2], w, ws, x_scale=xs),
                lambda: lin(x, d8(64, 32).t(), ws, x_scale=xs),
                lambda: gat(x, w, d8(31, 64), ws, ws, x_scale=xs),
                lambda: gat(x, w, d8(32, 64, "pad"), ws, ws, x_scale=xs),   # other strides
                lambda: gat(x, w, w, ws, ws[:31], x_scale=xs),
                lambda: llar.quantize_rows(x),
                lambda: llar.quantize_rows(v.double()),
                lambda: llar.quantize_rows(v.cpu()),
                lambda: llar.quantize_rows(v[0, 0])):
        with pytest.raises((ValueError, TypeError, llar.LlarError)):
            bad()
