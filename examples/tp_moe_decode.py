"""A mixture-of-experts layer of tensor- or expert-parallel decoding on one GPU:
every emulated rank computes its share of the experts' blocks for the tokens of one
step, and the AllReduce sums the partial outputs.

    all:      weights, experts = the top_k of x router^T
    rank r:   p_r = sum over a token's experts of weight * (silu(x wg_r^T) * (x wu_r^T)) wd_r^T  [+ x on rank 0]
    all:      y = sum_r p_r                           (AllReduce)

--split inner: rank r holds inner / N of every expert's width (its sums are whole).
--split experts: rank r holds experts / N of the experts; the numbers of the others lie
outside its own and add nothing.  --int8: 8-bit weights with a scale for each output
channel, tokens and inner rows quantised on the way.

    python examples/tp_moe_decode.py [--ranks 8] [--hidden 4096] [--inner 8192] [--experts 64] [--top-k 8]
                                     [--tokens 1] [--split inner|experts] [--int8] [--steps 100]

prints the difference from the same layer on one rank in binary32, relative to its result
(tokens and what the layer adds to them), and the time of a pass.
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import message_allreduce_amd as llar


class Layer:
    """The layer's weights, split over the ranks, and a communicator for its outputs."""

    def __init__(self, ranks, hidden, inner, experts, top_k, tokens, split="inner", int8=False, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape):
            return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0, shape[-1] ** -0.5, generator=gen)

        self.ranks, self.top_k, self.experts, self.split, self.int8 = ranks, top_k, experts, split, int8
        self.router = normal(experts, hidden)
        whole = {"gate": normal(experts, inner, hidden), "up": normal(experts, inner, hidden),
                 "down": normal(experts, hidden, inner)}
        self.whole = whole
        self.parts = []
        for r in range(ranks):
            if split == "inner":
                p = slice(inner * r // ranks, inner * (r + 1) // ranks)
                part = {"w_gate": whole["gate"][:, p], "w_up": whole["up"][:, p], "w_down": whole["down"][:, :, p]}
            else:
                p = slice(experts * r // ranks, experts * (r + 1) // ranks)
                part = {"w_gate": whole["gate"][p], "w_up": whole["up"][p], "w_down": whole["down"][p]}
            if int8:
                for name in ("gate", "up", "down"):
                    part["w_" + name], part[name + "_scale"] = llar.quantize_rows(part["w_" + name].contiguous())
            self.parts.append((p.start, part))
        self.comm = llar.Communicator(ranks, dtype, tokens * hidden * self.router.element_size())

    def forward(self, x):
        weights, experts = llar.moe_route(x, self.router, self.top_k)
        partials = []
        for r, (first, part) in enumerate(self.parts):
            mine = experts if self.split == "inner" else experts - first
            partials.append(llar.moe_ffn(x, mine, weights, residual=x if r == 0 else None, **part))
        y = torch.empty_like(x)
        self.comm.allreduce(partials, y)
        return y

    def reference(self, x):
        """The layer on one rank in binary32, by torch, with the unquantised weights."""
        logits = x.double() @ self.router.double().t()
        top = logits.topk(self.top_k, dim=1)
        weights, experts = torch.softmax(top.values, 1).float(), top.indices
        xf = x.float()
        y = xf.clone()
        for e in range(self.experts):
            weight = torch.where(experts == e, weights, torch.zeros_like(weights)).sum(1, keepdim=True)
            g, u, d = (self.whole[name][e].float() for name in ("gate", "up", "down"))
            y += weight * ((torch.nn.functional.silu(xf @ g.t()) * (xf @ u.t())) @ d.t())
        return y

    def close(self):
        self.comm.close()


def run(ranks, hidden, inner, experts, top_k, tokens, split="inner", int8=False, steps=0):
    """(device status, difference of the results in the 2-norm relative to theirs, x included, seconds a pass)."""
    layer = Layer(ranks, hidden, inner, experts, top_k, tokens, split, int8)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    y, want = layer.forward(x), layer.reference(x)
    off = ((y.float() - want).norm() / want.norm()).item()
    status, _ = layer.comm.device_status()
    took = None
    if steps:
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(steps):
            layer.forward(x)
        torch.cuda.synchronize()
        took = (time.perf_counter() - t) / steps
    layer.close()
    return status, off, took


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=8192)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--split", choices=["inner", "experts"], default="inner")
    ap.add_argument("--int8", action="store_true")
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    status, off, took = run(a.ranks, a.hidden, a.inner, a.experts, a.top_k, a.tokens, a.split, a.int8, a.steps)
    print("device status %d; off by (2-norm): %.2g" % (status, off))
    print("forward: %.1f us, all %d ranks one after another" % (took * 1e6, a.ranks))
    return 1 if status or off > (0.04 if a.int8 else 0.02) else 0


if __name__ == "__main__":
    sys.exit(main())
