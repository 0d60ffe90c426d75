"""The mixture-of-experts layer of examples/tp_moe_decode.py: router, experts and the
AllReduce together, against the same layer on one rank in binary32; and a block of
8-bit products with its AllReduce.

Tensors between two operators are bfloat16 (relative rounding at most 2^-8, about
2^-9.8 in the 2-norm): the inner rows, the partials and their sum, three in a row, stay
below 2^-8 in the 2-norm of the whole.  8-bit: a row of normal values has its largest at
3 to 4.5 standard deviations, so a quantised value is off by about 4.5 / 127 / sqrt(12) =
1.0 % of one deviation.  Both factors of the three products are quantised: the gate's and
the up's product are each off by 1.4 %, their product with the activation by 2.5 % at
most, the last product by 1.4 % more of its own: 2.9 % of what the layer adds, which is
less than the residual it is added to."""
import os
import sys

import pytest
import torch

import message_allreduce_amd as llar

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("split", ["inner", "experts"])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("ranks,hidden,inner,experts,top_k,tokens", [(8, 1024, 512, 16, 4, 1), (4, 512, 264, 8, 2, 37),
                                                                     (2, 264, 96, 6, 6, 70), (3, 128, 100, 10, 1, 5)])
def test_layer_matches_one_rank(ranks, hidden, inner, experts, top_k, tokens, int8, split):
    import tp_moe_decode
    status, off, _ = tp_moe_decode.run(ranks, hidden, inner, experts, top_k, tokens, split, int8)
    assert status == 0
    assert off < (0.03 if int8 else 2.0 ** -8), off


@pytest.mark.parametrize("tokens", [1, 12, 40])
def test_block_of_8_bit_products(tokens):
    """The gated block and the row-parallel product in 8 bits, split over ranks, summed by the AllReduce: what
    the products' values give in binary64, with three bfloat16 roundings (h, partials, their sum)."""
    ranks, hidden, inner = 4, 512, 1024
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)

    def normal(rows, cols):
        return torch.empty(rows, cols, device="cuda").normal_(0, cols ** -0.5, generator=gen)

    x = torch.empty(tokens, hidden, device="cuda").normal_(generator=gen).bfloat16()
    comm = llar.Communicator(ranks, torch.bfloat16, tokens * hidden * 2)
    partials, want = [], x.double()
    for r in range(ranks):
        wg, gs = llar.quantize_rows(normal(inner // ranks, hidden))
        wu, us = llar.quantize_rows(normal(inner // ranks, hidden))
        wd, ds = llar.quantize_rows(normal(hidden, inner // ranks))
        h = llar.gated_ffn_int8(x, wg, wu, gs, us)
        partials.append(llar.linear_int8(h, wd, ds, residual=x if r == 0 else None))
        q, s = llar.quantize_rows(x)
        X = q.double() * s.double()[:, None]
        g, u = ((X @ w.double().t().contiguous()) * sc.double() for w, sc in ((wg, gs), (wu, us)))
        hq, hs = llar.quantize_rows(h)
        assert (h.double() - g * torch.sigmoid(g) * u).norm() < 2.0 ** -8 * h.double().norm()
        want = want + ((hq.double() * hs.double()[:, None]) @ wd.double().t().contiguous()) * ds.double()
    y = torch.empty_like(x)
    comm.allreduce(partials, y)
    assert comm.device_status()[0] == 0
    comm.close()
    assert (y.double() - want).norm() < 2.0 ** -8 * want.norm()
