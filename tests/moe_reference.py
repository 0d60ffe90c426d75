"""Experts' layers of any size with their definition in binary64, on any device, and how far a result may be from it.

A token's result is compared in the 2-norm: with `half` the largest error that rounding a value once to the output's
type can make (half a step there), what |y - want| exceeds `half` by, element by element, is what the sums behind the
rounding are off by at the least.  Its norm over a token's outputs may be

- (2.5 sqrt(k) + sqrt(n top_k) + 48) 2^-24 of the result's norm: a sum of N terms of random signs makes N roundings of
  2^-24 at most of partial sums whose squares grow evenly to the result's, 0.41 sqrt(N) 2^-24 of it in the 2-norm
  (two sums over k feed an inner value, one over n and the choices follows; the rest is slack of 2.4 to 4, and what
  the activation, weights and scales round, an 8-bit row's scale like its largest value);
- and 2^-17 for the activation's exponential where results have 16 bits;
- and what the inner rows round: two bfloat16 numbers 2^-16, two binary16 ones 2^-22 (values of 2^-3 and more);
- 8-bit: an inner value next to a half may take the other whole number, one step times its row of weights.

Routing weights are 0.5 .. 1.5 in magnitude, so that a choice that is left out cannot hide.
"""
import math

import torch

# tokens, k, n, outputs, experts, top_k: few outputs and many choices or long inner rows, also a batch's last tokens alone
SHARED = [(59, 79, 227, 479, 94, 8), (16, 64, 1000, 24, 128, 4), (30, 40, 600, 130, 200, 6), (1, 64, 9000, 40, 40, 32),
          (67, 40, 520, 72, 300, 5), (65, 40, 8000, 33, 24, 16), (64, 1032, 520, 264, 6, 2), (3, 520, 264, 520, 12, 4),
          (40, 72, 200, 6161, 3, 2), (5, 136, 2400, 6200, 5, 3)]
# a rank's layers, where a wave takes many steps of k and crosses experts
WIDE = [(m, *layer) for layer in ((4096, 1024, 4096, 64, 8), (8192, 3584, 8192, 8, 2)) for m in (1, 16, 64)]

EXTRA = {torch.float32: 0.0, torch.float16: 2.0 ** -17 + 2.0 ** -22, torch.bfloat16: 2.0 ** -17 + 2.0 ** -16}


class Layer:
    """Inputs of a call.  size: tokens, k, inner width n, outputs, experts, top_k."""

    def __init__(self, size, dtype, int8=False, device="cuda", seed=0):
        self.size, self.dtype, self.int8 = size, dtype, int8
        m, k, n, outs, count, top_k = size
        g = torch.Generator(device=device)
        g.manual_seed(seed + sum(size))

        def weights(rows, cols):
            if not int8:
                return torch.empty(count, rows, cols, dtype=dtype, device=device).normal_(0, cols ** -0.5, generator=g), None
            q = torch.empty(count, rows, cols, dtype=torch.int8, device=device)
            for e in range(count):
                q[e] = torch.empty(rows, cols, device=device).normal_(0, 32, generator=g).round_().clamp_(-127, 127)
            return q, torch.empty(count, rows, device=device).uniform_(0.8, 1.25, generator=g) * (cols ** -0.5 / 32)

        self.x = torch.empty(m, k, dtype=dtype, device=device).normal_(generator=g)
        (self.gate, self.gate_scale), (self.up, self.up_scale), (self.down, self.down_scale) = (
            weights(n, k), weights(n, k), weights(outs, n))
        if top_k <= count:
            self.experts = torch.rand(m, count, generator=g, device=device).argsort(1)[:, :top_k].int().contiguous()
        else:
            self.experts = torch.randint(0, count, (m, top_k), generator=g, device=device).int()
        w = torch.rand(m, top_k, generator=g, device=device) + 0.5
        self.weights = torch.where(torch.rand(m, top_k, generator=g, device=device) < 0.5, -w, w)

    def call(self, **more):
        import message_allreduce_amd as llar
        scales = {"gate_scale": self.gate_scale, "up_scale": self.up_scale, "down_scale": self.down_scale} if self.int8 else {}
        return llar.moe_ffn(self.x, self.experts, self.weights, self.gate, self.up, self.down, **scales, **more)


def rows_quantized(t):
    top = t.abs().amax(1, keepdim=True)
    s = (top / 127).float().double()
    return torch.round(t / torch.where(s > 0, s, 1.0)).clamp(-127, 127) * (s > 0), s


def definition(layer, gone=None, inner=None):
    """(want, flips): the result, and what inner values next to a half may add to a token's norm.  Mistakes to be
    found: gone, (expert, first, last), inner columns left out of the second product; inner, the type that inner
    rows are rounded to."""
    m, k, n, outs, count, top_k = layer.size
    x = layer.x.double()
    want = torch.zeros(m, outs, dtype=torch.float64, device=x.device)
    flips = torch.zeros(m, dtype=torch.float64, device=x.device)
    if layer.int8:
        x, xs = rows_quantized(x)
    for e in layer.experts.unique().tolist():
        if not 0 <= e < count:
            continue
        here = layer.experts == e
        token = here.any(1).nonzero()[:, 0]
        a = torch.where(here, layer.weights, 0.0).double().sum(1)[token][:, None]

        def product(rows, name):
            w = getattr(layer, name)[e].double()
            if layer.int8:
                w = w * getattr(layer, name + "_scale")[e].double()[:, None]
            return torch.mm(rows, w.t().contiguous()), w

        g, u = product(x[token], "gate")[0], product(x[token], "up")[0]
        if layer.int8:
            g, u = g * xs[token], u * xs[token]
        h = g * torch.sigmoid(g) * u
        if layer.int8:
            q, s = rows_quantized(h)
            steps = h / s
            # h is off by at most 19 roundings of binary32 (3 in g and in u, 8 in the activation of slope 1.2, 3
            # in their product and its row), s by one more
            near = (steps - torch.floor(steps) - 0.5).abs() <= 40 * steps.abs() * 2.0 ** -24
            h = q * s
        if inner:
            h = h.to(inner).double()
        if gone and gone[0] == e:
            h[:, gone[1]:gone[2]] = 0
        y, w = product(h, "down")
        want.index_add_(0, token, a * y)
        if layer.int8:
            flips.index_add_(0, token, (near * s * a.abs() * w.norm(dim=0)).sum(1))
    return want, flips


def half_step(want, dtype):
    info = torch.finfo(dtype)
    exponent = torch.frexp(want)[1].double() - 1
    return torch.exp2(exponent.clamp(min=math.log2(info.smallest_normal))) * (info.eps / 2)


def beyond(y, want, dtype):
    """Of every token, the norm of what its result is off by beyond one rounding."""
    return ((y.double() - want).abs() - half_step(want, dtype)).clamp(min=0).norm(dim=1)


def allowed(layer, want, flips):
    m, k, n, outs, count, top_k = layer.size
    sums = (2.5 * math.sqrt(k) + math.sqrt(n * top_k) + 48) * 2.0 ** -24
    return (sums + (0.0 if layer.int8 else EXTRA[layer.dtype])) * want.norm(dim=1) + flips
