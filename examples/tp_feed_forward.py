"""A tensor-parallel feed-forward layer on one GPU: every emulated rank computes
its share with the library's operators, and the AllReduce sums the partial
outputs.

    rank r:   h_r = silu(x wg_r^T) * (x wu_r^T)       (column-parallel: wg_r, wu_r hold inner / N rows)
              p_r = h_r wd_r^T  [+ x on rank 0]       (row-parallel, the residual in the epilogue)
    all:      y = sum_r p_r                           (AllReduce)

and back: dh_r, dwd_r from dy; dx_r, dwg_r, dwu_r from dh_r; dx = dy + sum_r dx_r.

    python examples/tp_feed_forward.py [--ranks 8] [--hidden 8192] [--inner 28672] [--tokens 1] [--steps 100]

prints the largest difference from the same layer on one rank in binary32 and
the time of a forward and of a forward and backward pass.
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

    def __init__(self, ranks, hidden, inner, tokens, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(rows, cols):
            return torch.empty(rows, cols, dtype=dtype, device="cuda").normal_(0, cols ** -0.5, generator=gen)

        self.ranks, self.wg, self.wu, self.wd = ranks, normal(inner, hidden), normal(inner, hidden), normal(hidden, inner)
        self.part = [slice(inner * r // ranks, inner * (r + 1) // ranks) for r in range(ranks)]
        self.comm = llar.Communicator(ranks, dtype, tokens * hidden * self.wg.element_size())

    def forward(self, x, save=False):
        """(y, what the backward pass needs)."""
        partials, saved = [], []
        for r, p in enumerate(self.part):
            gate = up = None
            h = llar.gated_ffn(x, self.wg[p], self.wu[p], save=save)
            if save:
                h, gate, up = h
            saved.append((h, gate, up))
            # a rank's columns of wd are a slice of its rows: no copy
            partials.append(llar.linear(h, self.wd[:, p], residual=x if r == 0 else None))
        y = torch.empty_like(x)
        self.comm.allreduce(partials, y)
        return y, saved

    def backward(self, dy, x, saved):
        """(dx, [(dwg, dwu, dwd) of every rank])."""
        partials, grads = [], []
        for p, (h, gate, up) in zip(self.part, saved):
            dh, dwd, _ = llar.linear_backward(dy, h, self.wd[:, p])
            dx, dwg, dwu = llar.gated_ffn_backward(dh, x, self.wg[p], self.wu[p], gate, up)
            partials.append(dx)
            grads.append((dwg, dwu, dwd))
        dx = torch.empty_like(x)
        self.comm.allreduce(partials, dx)
        return dx.add_(dy), grads

    def reference(self, x, dy=None):
        """The layer on one rank in binary32, by torch: y, and with dy (dx, dwg, dwu, dwd)."""
        x, wg, wu, wd = (t.float().requires_grad_(dy is not None) for t in (x, self.wg, self.wu, self.wd))
        y = x + (torch.nn.functional.silu(x @ wg.t()) * (x @ wu.t())) @ wd.t()
        if dy is None:
            return y
        return y.detach(), torch.autograd.grad(y, (x, wg, wu, wd), dy.float())

    def close(self):
        self.comm.close()


def off(got, want):
    """Relative difference in the 2-norm."""
    return ((got.float() - want).norm() / want.norm()).item()


def run(ranks, hidden, inner, tokens, steps=0):
    layer = Layer(ranks, hidden, inner, tokens)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    dy = torch.randn(tokens, hidden, device="cuda").bfloat16()
    y, saved = layer.forward(x, save=True)
    dx, grads = layer.backward(dy, x, saved)
    want, (wdx, wdwg, wdwu, wdwd) = layer.reference(x, dy)
    worst = {"y": off(y, want), "dx": off(dx, wdx), "dwg": off(torch.cat([g[0] for g in grads]), wdwg),
             "dwu": off(torch.cat([g[1] for g in grads]), wdwu), "dwd": off(torch.cat([g[2] for g in grads], 1), wdwd)}
    status, _ = layer.comm.device_status()
    times = {}
    if steps:
        def both():
            out, kept = layer.forward(x, save=True)
            layer.backward(dy, x, kept)
        for name, f in (("forward", lambda: layer.forward(x)), ("forward and backward", both)):
            f()
            torch.cuda.synchronize()
            t = time.perf_counter()
            for _ in range(steps):
                f()
            torch.cuda.synchronize()
            times[name] = (time.perf_counter() - t) / steps
    layer.close()
    return status, worst, times


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--inner", type=int, default=28672)
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    status, worst, times = run(a.ranks, a.hidden, a.inner, a.tokens, a.steps)
    print("device status %d; off by (2-norm): %s" % (status, ", ".join("%s %.2g" % kv for kv in worst.items())))
    for name, t in times.items():
        print("%s: %.1f us, all %d ranks one after another" % (name, t * 1e6, a.ranks))
    return 1 if status or max(worst.values()) > 0.02 else 0


if __name__ == "__main__":
    sys.exit(main())
