"""The mixture-of-experts operators against their definitions in binary64.

Tolerances.  Routing: the choice is exact, a weight is binary64's rounded once.
Experts, with u the I/O type's unit roundoff: the two products and the activation
are off as in test_gpu_ffn.gated_case; an inner row rounds to the I/O type (u);
the second product and the weighted sum add (n top_k + 16) 2^-23 of their absolute
values; the output rounds once.  8-bit: both first products are exact whole sums
with three roundings each; a quantised inner value differs from the definition's
only where that is as near to a half as its own error is large, by one step.
"""
import math

import pytest
import torch

import message_allreduce_amd as llar
from test_gpu_ffn import DTYPES, EPS, TINY, U, Draw, act64, check, ids, mm64
from test_gpu_int8 import Draw8, quantized64

pytestmark = pytest.mark.gpu


# ---- routing ---------------------------------------------------------------------------

def route64(x, router, top_k, scoring, normalize):
    logits = mm64(x.double(), router.double().t())
    order = torch.sort(torch.nan_to_num(logits, nan=-math.inf, posinf=math.inf, neginf=-math.inf), dim=1, descending=True,
                       stable=True).indices[:, :top_k]
    score = torch.softmax(logits, 1) if scoring == "softmax" else torch.sigmoid(logits)
    w = score.gather(1, order)
    return (w / w.sum(1, keepdim=True) if normalize else w), order


def route_case(x, router, top_k, scoring="softmax", normalize=True):
    w, e = llar.moe_route(x, router, top_k, scoring=scoring, normalize=normalize)
    assert w.dtype == torch.float32 and e.dtype == torch.int32 and w.shape == e.shape == (*x.shape[:-1], top_k)
    want, order = route64(x, router, top_k, scoring, normalize)
    assert torch.equal(e.long(), order), (e.long() != order).nonzero()[:3].tolist()
    off = (w.double() - want).abs() - (1.01 * 2.0 ** -24 + 1e-11) * want.abs() - 2.0 ** -149
    assert (off <= 0).all(), off.max().item()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_route_sizes(normalize, scoring, dtype):
    for m, experts, k, top_k in ((1, 1, 1, 1), (1, 8, 64, 2), (1, 64, 4096, 8), (3, 5, 77, 5), (16, 16, 130, 4), (17, 33, 65, 1),
                                 (64, 256, 520, 8), (5, 1024, 96, 32), (100, 160, 2048, 6), (2, 65, 8200, 3)):
        d = Draw(m + experts + k, dtype)
        route_case(d(m, k), d(experts, k, scale=2 * k ** -0.5), top_k, scoring, normalize)
    for layout in ("pad", "off"):
        d = Draw(7, dtype)
        route_case(d(9, 71, layout), d(40, 71, layout, 0.2), 4, scoring, normalize)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_route_takes_the_lowest_of_equals(dtype):
    d = Draw(3, dtype)
    x, r = d(20, 64), d(70, 64, scale=0.2)
    r[40:] = r[:30]           # every one of these twice
    r[33] = r[31]
    route_case(x, r, 12)
    w, e = llar.moe_route(x, torch.zeros_like(r), 6)
    assert torch.equal(e, torch.arange(6, device="cuda", dtype=torch.int32).expand(20, 6)) and (w * 6 - 1).abs().max() < 1e-6
    # products that differ only beyond binary32: 1 and 1 + 2^-40
    if dtype == torch.float32:
        x = torch.tensor([[1.0, 2.0 ** -40]], device="cuda")
        r = torch.tensor([[1.0, 0.0], [1.0, 1.0], [1.0, -1.0]], device="cuda")
        assert llar.moe_route(x, r, 3)[1].tolist() == [[1, 0, 2]]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_route_with_infinities_and_nans(dtype):
    """Choices are distinct experts whatever the logits are; other tokens see nothing of it."""
    d = Draw(4, dtype)
    x, r = d(6, 64), d(20, 64, scale=0.2)
    clean = llar.moe_route(x, r, 4)
    x[1, 3], x[2, 5], x[4] = math.nan, math.inf, math.inf
    w, e = llar.moe_route(x, r, 4)
    assert w[1].isnan().all() and e[1].tolist() == [0, 1, 2, 3]
    for t in range(6):
        assert len(set(e[t].tolist())) == 4 and 0 <= e[t].min() and e[t].max() < 20
        if t in (0, 3, 5):
            assert torch.equal(w[t], clean[0][t]) and torch.equal(e[t], clean[1][t])
    r[7, 0] = math.nan        # one expert's logit for every token: below all others
    w, e = llar.moe_route(d(5, 64), r, 19)
    assert (e != 7).all() and w.isnan().all()
    big = torch.full((1, 8), 60000.0 if dtype == torch.float16 else 1e30, dtype=dtype, device="cuda")
    w, e = llar.moe_route(big, big.expand(3, 8) * torch.tensor([[1.0], [-1.0], [0.5]], dtype=dtype, device="cuda"), 2)
    assert e.tolist() == [[0, 2]] and w.tolist() == [[1.0, 0.0]]
    w, e = llar.moe_route(big, big.expand(3, 8) * torch.tensor([[1.0], [-1.0], [0.5]], dtype=dtype, device="cuda"), 3,
                          scoring="sigmoid", normalize=False)
    assert e.tolist() == [[0, 2, 1]] and w.tolist() == [[1.0, 1.0, 0.0]]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_route_shapes(dtype):
    d = Draw(5, dtype)
    x, r = d(6, 40), d(12, 40)
    w, e = llar.moe_route(x, r, 3)
    w3, e3 = llar.moe_route(x.view(2, 3, 40), r, 3)
    assert torch.equal(w3.view(6, 3), w) and torch.equal(e3.view(6, 3), e)
    w1, e1 = llar.moe_route(x[2], r, 3)
    assert torch.equal(w1, w[2]) and torch.equal(e1, e[2])
    assert torch.equal(llar.moe_route(x[1:2].expand(4, 40), r, 3)[1], e[1:2].expand(4, 3))
    empty = lambda *s: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    assert llar.moe_route(empty(0, 40), r, 3)[0].shape == (0, 3)
    assert llar.moe_route(x, r, 0)[1].shape == (6, 0)
    w, e = llar.moe_route(empty(2, 0), empty(4, 0), 2, normalize=False)
    assert e.tolist() == [[0, 1]] * 2 and w.tolist() == [[0.25, 0.25]] * 2


# ---- experts -----------------------------------------------------------------------------

class Weights:
    """E experts' matrices.  layout: "row" (dense), "halves" (gate and up are halves of one buffer), "pad" (rows of
    wider buffers), "off" (unaligned)."""

    def __init__(self, seed, dtype, experts, n, k, outs, int8=False, layout="row"):
        d, d8 = Draw(seed, dtype), Draw8(seed)

        def one(rows, cols):
            wide = {"pad": 16, "off": 3}.get(layout, 0)
            if int8:
                t = d8(max(experts * rows, 1), cols + wide)[:experts * rows]
            else:
                t = d(max(experts * rows, 1), cols + wide, scale=max(cols, 1) ** -0.5)[:experts * rows]
            t = t.view(experts, rows, cols + wide)
            return t[:, :, 1:cols + 1] if layout == "off" else t[:, :, :cols]

        if layout == "halves":
            both = one(2 * n, k)
            self.gate, self.up = both[:, :n], both[:, n:]
        else:
            self.gate, self.up = one(n, k), one(n, k)
        self.down = one(outs, n)
        self.scales = {}
        if int8:
            def s(rows, cols):
                return d8.scales(experts * rows, cols).view(experts, rows)
            self.scales = {"gate_scale": s(n, k), "up_scale": s(n, k), "down_scale": s(outs, n)}

    def call(self, x, experts, weights, **more):
        return llar.moe_ffn(x, experts, weights, self.gate, self.up, self.down, **self.scales, **more)


def moe64(x, experts, weights, w, act, dtype):
    """The definition, and what the kernels' sums may be off before the output's rounding."""
    m, (count, n, k), outs = x.shape[0], w.gate.shape, w.down.shape[1]
    y = torch.zeros(m, outs, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(y)
    total = torch.zeros_like(y)
    int8 = bool(w.scales)
    X = x.double()
    if int8:
        X, xs = quantized64(x)
        xs = xs.double()[:, None]
    for e in range(count):
        weight = torch.where(experts == e, weights, torch.zeros_like(weights)).double()
        token = (experts == e).any(1).nonzero()[:, 0]
        if token.numel() == 0:
            continue
        a = weight.sum(1)[token][:, None]
        aa = weight.abs().sum(1)[token][:, None]
        rows = X[token]
        g, u = mm64(rows, w.gate[e].double().t()), mm64(rows, w.up[e].double().t())
        if int8:
            g = g * xs[token] * w.scales["gate_scale"][e].double()
            u = u * xs[token] * w.scales["up_scale"][e].double()
            ge, ue = 3.03 * 2.0 ** -24 * g.abs(), 3.03 * 2.0 ** -24 * u.abs()
        else:
            ge = (k + 16) * EPS * mm64(rows.abs(), w.gate[e].double().t().abs())
            ue = (k + 16) * EPS * mm64(rows.abs(), w.up[e].double().t().abs())
        v = act64(g, act)
        ve = 1.2 * ge + 16 * EPS * v.abs()
        h, he = v * u, ve * u.abs() + v.abs() * ue + ve * ue + EPS * (v * u).abs()
        down = w.down[e].double()
        if int8:
            down = down * w.scales["down_scale"][e].double()[:, None]
            q, hs = quantized64(h)
            s = hs.double()[:, None]
            top = h.abs().amax(1, keepdim=True) if n else s
            some = s > 0
            rel = torch.where(some, he.amax(1, keepdim=True) / torch.where(some, top, torch.ones_like(top)), s) + 2.0 ** -23 \
                if n else s
            steps = h / torch.where(some, s, torch.ones_like(s))
            near = ((steps - torch.floor(steps) - 0.5).abs() <= he / torch.where(some, s, torch.ones_like(s)) + 130 * rel)
            he = q.abs() * s * rel + torch.where(near & some, 1.01 * s, torch.zeros_like(s))
            h = q * s
        else:
            # rounded once; fp16: and what that left lifted by 2^11 and rounded
            he = he + (1.01 * U[dtype] ** 2 * h.abs() + TINY[dtype] * 2.0 ** -11 if dtype == torch.float16 else
                       1.01 * U[dtype] * h.abs() + TINY[dtype])
        part = mm64(h, down.t())
        size = mm64(h.abs(), down.t().abs())
        y.index_add_(0, token, a * part)
        err.index_add_(0, token, aa * (mm64(he, down.t().abs()) + 4 * EPS * size))
        total.index_add_(0, token, aa * size)
    return y, err + (n * experts.shape[1] + 16) * EPS * total


def choose(seed, m, count, top_k, away=0.0, twice=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    e = torch.rand(m, max(count, 1), generator=g, device="cuda").argsort(1)[:, :top_k].int()
    if e.shape[1] < top_k or twice:  # more choices than experts: some twice
        e = torch.randint(0, max(count, 1), (m, top_k), generator=g, device="cuda").int()
    w = torch.randn(m, top_k, generator=g, device="cuda")
    if away:
        gone = torch.rand(m, top_k, generator=g, device="cuda") < away
        e = torch.where(gone, torch.where(w > 0, -1, count + 7).int(), e)
    return e.contiguous(), w


def moe_case(m, k, n, outs, count, top_k, dtype, act="silu", int8=False, residual=False, layout="row", xl="row", away=0.0,
             twice=False, wide_ids=False, seed=0):
    w = Weights(seed + 31 * m + n + k, dtype, count, n, k, outs, int8, layout)
    d = Draw(seed + m, dtype)
    x, r = d(m, k, xl), d(m, outs) if residual else None
    e, a = choose(seed + m + count, m, count, top_k, away, twice)
    y = w.call(x, e.long() if wide_ids else e, a, activation=act, residual=r)
    assert y.shape == (m, outs) and y.dtype == dtype
    want, err = moe64(x, e, a, w, act, dtype)
    if residual:
        want = want + r.double()
        err = err + EPS * (want.abs() + r.double().abs())
    check(y, want, err, "moe %s" % ((m, k, n, outs, count, top_k, dtype, act, int8, layout, xl),))


# tokens, k, n, outputs, experts, top_k: fewer and more choices than experts, one block of 16 tokens and four, more than 64
SIZES = [(1, 1, 1, 1, 1, 1), (1, 64, 32, 64, 8, 2), (2, 96, 400, 64, 8, 4), (1, 256, 96, 200, 64, 8), (2, 77, 45, 33, 5, 3), (3, 520, 264, 520, 12, 4),
         (7, 64, 128, 64, 3, 3), (16, 128, 64, 130, 8, 2), (17, 130, 72, 64, 40, 2), (32, 64, 48, 96, 4, 1), (33, 96, 80, 40, 16, 4),
         (48, 200, 100, 72, 8, 2), (64, 64, 33, 48, 100, 8), (64, 1032, 520, 264, 6, 2), (65, 72, 40, 64, 8, 2), (150, 64, 64, 40, 24, 3)]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, int8, dtype):
    moe_case(*size, dtype, int8=int8)
    moe_case(*size, dtype, "gelu", int8=int8, residual=True, away=0.4, seed=1)


# many outputs: 32 columns a workgroup in the second kernel
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("m", [3, 5, 20, 40, 64])
def test_wide_outputs(m, int8, dtype):
    moe_case(m, 72, 56, 6200, 5, 2, dtype, int8=int8, residual=True)
    moe_case(m, 72, 200, 6161, 3, 1, dtype, int8=int8, away=0.2)


# few outputs and many experts: a column tile's experts shared between workgroups, also of a batch's last tokens alone
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("size", [(59, 79, 227, 479, 94, 8), (16, 64, 1000, 24, 128, 4), (30, 40, 600, 130, 200, 6), (1, 64, 9000, 40, 40, 32),
                                  (67, 40, 520, 72, 300, 5), (65, 40, 8000, 33, 24, 16)], ids=str)
def test_many_experts_few_outputs(size, int8, dtype):
    moe_case(*size, dtype, int8=int8, residual=True)
    moe_case(*size, dtype, int8=int8, away=0.5, twice=True)


# rows that a kernel's own workgroups quantise, and just beyond
@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_rows_quantized_on_the_way(dtype):
    for size in ((1, 8192, 40, 24, 4, 2), (2, 8200, 40, 24, 4, 2), (2, 8191, 33, 40, 4, 3), (1, 100, 2047, 40, 16, 8),
                 (1, 64, 2049, 40, 16, 8), (2, 40, 1000, 40, 8, 8), (16, 64, 256, 40, 8, 4), (16, 64, 257, 40, 8, 4),
                 (17, 64, 64, 40, 8, 1), (13, 64, 40, 6200, 8, 5)):
        moe_case(*size, dtype, int8=True, away=0.2)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("layout", ["row", "halves", "pad", "off"])
def test_layouts_and_activations(layout, int8, dtype):
    for act in ("none", "relu", "gelu", "gelu_tanh", "silu"):
        for size in ((1, 71, 45, 64, 8, 3), (5, 136, 72, 40, 4, 2), (40, 45, 33, 71, 6, 2)):
            moe_case(*size, dtype, act, int8, layout=layout)
    for xl in ("pad", "off"):
        moe_case(9, 71, 45, 33, 8, 2, dtype, int8=int8, layout=layout, xl=xl, wide_ids=True)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
def test_choices(int8, dtype):
    """The same expert twice, everyone the same one, as many as there may be, numbers beyond the experts."""
    moe_case(6, 64, 48, 40, 3, 5, dtype, int8=int8, twice=True, away=0.2)
    moe_case(40, 64, 48, 40, 4, 6, dtype, int8=int8, twice=True)
    moe_case(64, 40, 24, 40, 1024, 32, dtype, int8=int8)
    moe_case(3, 40, 24, 40, 1024, 32, dtype, int8=int8, away=0.5)
    w = Weights(1, dtype, 9, 48, 64, 40, int8)
    x = Draw(2, dtype)(50, 64)
    same = torch.full((50, 2), 4, dtype=torch.int32, device="cuda")
    a = torch.rand(50, 2, device="cuda")
    a[:, 1] = -0.5
    want, err = moe64(x, same, a, w, "silu", dtype)
    check(w.call(x, same, a), want, err, "one expert")
    far = torch.tensor([[-1, 9], [1 << 40, 2], [-(1 << 40), 1 << 31], [3, (1 << 32) + 3]], device="cuda")
    a = torch.rand(4, 2, device="cuda")
    a[0, 0] = math.nan  # the weight of no expert
    y = w.call(x[:4], far, a)
    assert (y[0] == 0).all() and (y[2] == 0).all()
    assert torch.equal(y[1], w.call(x[1:2], far[1:2, 1:].contiguous(), a[1:2, 1:].contiguous())[0])
    assert torch.equal(y[3], w.call(x[3:4], far[3:4, :1].contiguous(), a[3:4, :1].contiguous())[0])


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_small_values_are_not_lost(dtype):
    """Subnormal inputs and weights, and products of them that only the last weight makes large again."""
    tiny = torch.finfo(dtype).smallest_normal
    eps = torch.finfo(dtype).eps
    for m in (1, 20):
        w = Weights(1, dtype, 2, 16, 16, 16)
        for t in (w.gate, w.up, w.down):
            t.zero_()
        x = torch.zeros(m, 16, dtype=dtype, device="cuda")
        x[:, 0], x[:, 1] = tiny * eps * 3, 1.0            # subnormal in x
        w.gate[:, 0, 1] = 1.0
        w.up[:, 0, 0] = 1.0
        w.down[:, 0, 0] = 1.0
        w.gate[:, 1, 1] = 1.0
        w.up[:, 1, 1] = tiny * eps * 5                    # subnormal in a weight
        w.down[:, 1, 1] = 1.0
        w.gate[:, 2, 1] = w.up[:, 2, 1] = 1.0
        w.down[:, 2, 2] = tiny * eps * 7
        e, a = choose(1, m, 2, 1)
        a = torch.full_like(a, 1024.0)
        y = w.call(x, e, a, activation="relu")
        want = torch.tensor([3.0, 5.0, 7.0], device="cuda", dtype=torch.float64) * 1024 * tiny * eps
        assert torch.equal(y[:, :3].double(), want.expand(m, 3)), (y[0, :3].double() / (tiny * eps)).tolist()


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("m", [2, 24, 60])
def test_small_inner_rows_keep_their_digits(m, dtype):
    """Inner rows around 2^-19, where fp16 has five digits, whose sums large weights bring back into its range."""
    w = Weights(m, dtype, 6, 80, 72, 6200 if m == 24 else 96)
    x = Draw(m, dtype)(m, 72) * 2.0 ** -9
    e, a = choose(m, m, 6, 2)
    a = a * 2.0 ** 14
    check(w.call(x, e, a), *moe64(x, e, a, w, "silu", dtype), "inner rows of 2^-19, %d %s" % (m, dtype))


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
def test_what_is_not_finite_stays_with_its_tokens(int8, dtype):
    """A row of x, an expert's weights or scale, a routing weight: only the tokens that meet it see it."""
    for m in (6, 40):
        w = Weights(1, dtype, 8, 48, 64, 40, int8)
        x = Draw(2, dtype)(m, 64)
        e, a = choose(3, m, 8, 2)
        clean = w.call(x, e, a)
        x2, a2 = x.clone(), a.clone()
        x2[1, 3], x2[2, 60] = math.nan, math.inf
        a2[4, 0] = math.inf
        y = w.call(x2, e, a2)
        keep = [t for t in range(m) if t not in (1, 2, 4)]
        assert y[1].isnan().all() and not torch.isfinite(y[2]).any() and not torch.isfinite(y[4]).any()
        assert torch.equal(y[keep], clean[keep])
        if int8:
            w.scales["gate_scale"][5, 7] = math.nan
            w.scales["down_scale"][6, 3] = math.inf
        else:
            w.gate[5, 7, 1] = math.nan
            w.down[6, 3, 2] = math.inf
        y = w.call(x, e, a)
        five, six = (e == 5).any(1), (e == 6).any(1)
        assert y[five].isnan().all()
        other = ~(five | six)
        assert torch.equal(y[other], clean[other])
        only6 = six & ~five
        assert torch.equal(y[only6][:, [c for c in range(40) if c != 3]], clean[only6][:, [c for c in range(40) if c != 3]])


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
def test_zero_sizes(int8, dtype):
    def run(m, k, n, outs, count, top_k):
        w = Weights(1, dtype, count, n, k, outs, int8)
        e, a = choose(2, m, count, top_k)
        if count == 0:
            e = torch.zeros(m, top_k, dtype=torch.int32, device="cuda")
        r = torch.full((m, outs), 2.0, dtype=dtype, device="cuda")
        x = Draw(3, dtype)(max(m, 1), k)[:m]
        y = w.call(x, e, a, residual=r)
        assert y.shape == (m, outs) and (y == 2).all()
        y = w.call(x, e, a)
        assert y.shape == (m, outs) and (y == 0).all()
    for m in (3, 20, 70):
        run(m, 0, 8, 16, 4, 2)
        run(m, 8, 0, 16, 4, 2)
        run(m, 8, 16, 0, 4, 2)
        run(m, 8, 16, 24, 0, 2)
        run(m, 8, 16, 24, 4, 0)
    run(0, 8, 16, 24, 4, 2)


@pytest.mark.parametrize("int8", [False, True])
def test_shapes_outputs_and_residuals(int8):
    for m in (1, 2, 6, 40, 70):
        w = Weights(m, torch.bfloat16, 8, 48, 64, 40, int8)
        d = Draw(m, torch.bfloat16)
        x, r = d(m, 64), d(m, 40)
        e, a = choose(m, m, 8, 2)
        y = w.call(x, e, a, residual=r)
        if m % 2 == 0:
            y3 = w.call(x.view(2, -1, 64), e.view(2, -1, 2), a.view(2, -1, 2), residual=r.view(2, -1, 40))
            assert torch.equal(y3.view(m, 40), y)
        if m == 1:
            assert torch.equal(w.call(x[0], e[0], a[0], residual=r[0]), y[0])
        buf = torch.full((m + 2, 45), 9.0, dtype=torch.bfloat16, device="cuda")
        assert torch.equal(w.call(x, e, a, residual=r, out=buf[1:m + 1, 2:42]), y)
        buf[1:m + 1, 2:42] = 9.0
        assert (buf == 9).all()
        if int8:  # any strides
            assert torch.equal(w.call(x.t().contiguous().t(), e, a, residual=r), y)
        assert w.call(x, e, a, residual=r, out=r) is r and torch.equal(r, y)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
def test_long_batches_and_same_bits(int8, dtype):
    """More than 64 tokens are what 64 at a time are, and every call gives the same bits."""
    w = Weights(1, dtype, 12, 96, 128, 72, int8)
    x = Draw(2, dtype)(200, 128)
    e, a = choose(3, 200, 12, 3)
    y = w.call(x, e, a)
    for t in range(0, 200, 64):
        assert torch.equal(y[t:t + 64], w.call(x[t:t + 64], e[t:t + 64], a[t:t + 64]))
    for _ in range(3):
        assert torch.equal(w.call(x, e, a), y)


@pytest.mark.parametrize("int8", [False, True])
def test_another_stream_and_a_graph(int8):
    """Router and experts as a layer, on another stream and replayed with other tokens, other choices."""
    for m in (1, 5, 50):
        d = Draw(8, torch.bfloat16)
        x, router = d(m, 256), d(16, 256, scale=0.1)
        w = Weights(9, torch.bfloat16, 16, 128, 256, 256, int8)

        def layer(stream=None):
            a, e = llar.moe_route(x, router, 4, stream=stream)
            return w.call(x, e, a, residual=x, stream=stream)

        want = layer()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = layer(s)
        s.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer()
        for i in range(4):
            x.copy_(d(m, 256))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, layer()), (m, i)


def test_two_streams_at_once():
    """Calls that run at the same time have workspaces of their own."""
    w = Weights(1, torch.bfloat16, 16, 256, 512, 512)
    d = Draw(2, torch.bfloat16)
    xs = [d(24, 512) for _ in range(2)]
    es = [choose(i, 24, 16, 4) for i in range(2)]
    want = [w.call(x, *e) for x, e in zip(xs, es)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(w.call(xs[i], *es[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("int8", [False, True])
def test_experts_far_apart(int8):
    """Experts more than 2^31 elements apart, offsets beyond 2^32."""
    dtype = torch.int8 if int8 else torch.bfloat16
    n, k, outs, count, apart = 32, 64, 48, 3, (1 << 31) + 80
    big = torch.empty((count - 1) * apart + 100000, dtype=dtype, device="cuda")
    w = Weights(1, torch.bfloat16, count, n, k, outs, int8)
    far = Weights(1, torch.bfloat16, count, n, k, outs, int8)
    for i, name in enumerate(("gate", "up", "down")):
        t = getattr(w, name)
        f = big[i * 20000:].as_strided(t.shape, (apart, t.shape[2], 1))
        f.copy_(t)
        setattr(far, name, f)
    for m in (1, 20):
        x = Draw(2, torch.bfloat16)(m, k)
        e, a = choose(3, m, count, 2)
        assert torch.equal(far.call(x, e, a), w.call(x, e, a))


def test_refusals():
    d = Draw(1, torch.bfloat16)
    x, r = d(4, 64), d(8, 64)
    for bad in (lambda: llar.moe_route(x, r, 9),
                lambda: llar.moe_route(x, r, -1),
                lambda: llar.moe_route(x, d(8, 63), 2),
                lambda: llar.moe_route(x, r.float(), 2),
                lambda: llar.moe_route(x.cpu(), r, 2),
                lambda: llar.moe_route(x, r, 2, scoring="relu"),
                lambda: llar.moe_route(x, d(2000, 64), 2),
                lambda: llar.moe_route(x, d(64, 64), 33),
                lambda: llar.moe_route(d(64, 4).t(), r, 2),
                lambda: llar.moe_route(x, d(64, 8).t(), 2)):
        with pytest.raises((ValueError, TypeError, llar.LlarError)):
            bad()
    w, w8 = Weights(1, torch.bfloat16, 8, 32, 64, 40), Weights(1, torch.bfloat16, 8, 32, 64, 40, True)
    e, a = choose(1, 4, 8, 2)

    def call(x=x, e=e, a=a, w=w, **more):
        args = dict(w_gate=w.gate, w_up=w.up, w_down=w.down, **w.scales)
        args.update(more)
        return llar.moe_ffn(x, e, a, **args)

    call(), call(w=w8)
    for bad in (lambda: call(activation="swish"),
                lambda: call(x=x.float()),
                lambda: call(x=x.cpu()),
                lambda: call(x=d(4, 63)),
                lambda: call(x=d(64, 4).t()),
                lambda: call(e=e.float()),
                lambda: call(e=e.short()),
                lambda: call(e=e[:3]),
                lambda: call(e=e.repeat(1, 2)[:, ::2]),
                lambda: call(e=e.cpu()),
                lambda: call(a=a.double()),
                lambda: call(a=a[:, :1].contiguous()),
                lambda: call(a=a.bfloat16()),
                lambda: call(w_up=w.up[:, :31]),
                lambda: call(w_up=w.up[:7]),
                lambda: call(w_gate=w.gate.transpose(1, 2).contiguous().transpose(1, 2)),
                lambda: call(w_up=torch.cat([w.up, w.up], 2)[:, :, :64]),   # other strides
                lambda: call(w_down=w.down[:, :, :31].contiguous()),
                lambda: call(w_down=w8.down),
                lambda: call(w=w8, gate_scale=None),
                lambda: call(w=w8, up_scale=w8.scales["up_scale"][:, :31]),
                lambda: call(w=w8, down_scale=w8.scales["down_scale"].double()),
                lambda: call(w=w8, down_scale=w8.scales["down_scale"].t().contiguous().t()),
                lambda: call(gate_scale=w8.scales["gate_scale"]),
                lambda: call(residual=d(4, 39)),
                lambda: call(out=d(3, 40)),
                lambda: call(e=e.repeat(1, 20), a=a.repeat(1, 20))):
        with pytest.raises((ValueError, TypeError, llar.LlarError)):
            bad()
