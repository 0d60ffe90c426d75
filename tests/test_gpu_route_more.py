"""The router where logits are far below zero, and with more tokens than one launch has room for."""
import pytest
import torch

import message_allreduce_amd as llar
from test_gpu_ffn import DTYPES, ids
from test_gpu_moe import route64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("m", [1, 300])
def test_shares_of_far_sigmoids(m, dtype):
    """Sigmoids of -592 to -12000 have shares of their sum, though binary64 cannot hold the smaller ones."""
    x = torch.ones(m, 8, dtype=dtype, device="cuda")
    for first, step in ((-592, 4), (-600, 8), (-696, 4), (-704, 4), (-800, 4), (-12032, 64)):
        router = torch.zeros(6, 8, dtype=dtype, device="cuda")
        router[:, 2] = first - step * torch.tensor([2, 0, 1, 30, 3, 4], device="cuda")
        logits = router[:, 2].double()
        order = logits.sort(descending=True, stable=True).indices[:5]
        want = torch.softmax(logits[order], 0)  # s(l) = e^l here, to 2^-800
        w, e = llar.moe_route(x, router, 5, scoring="sigmoid")
        assert (e == order).all()
        off = (w.double() - want).abs() - (1.01 * 2.0 ** -24 + 1e-11) * want - 2.0 ** -149
        assert (off <= 0).all(), (first, w[0].tolist(), want.tolist())


def test_more_tokens_than_a_launch_has_waves():
    """65536 tokens at a time: both sides of the first border, beyond 2^26, and the last few."""
    m, k, experts = (1 << 26) + 300, 8, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.empty(m, k, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    router = torch.empty(experts, k, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w, e = llar.moe_route(x, router, 2)
    for at in (0, (1 << 16) - 500, (1 << 26) - 500, m - 700):
        part = slice(at, at + 700)
        want, order = route64(x[part], router, 2, "softmax", True)
        assert torch.equal(e[part].long(), order)
        assert ((w[part].double() - want).abs() <= (1.01 * 2.0 ** -24 + 1e-11) * want).all()
