"""The router where logits are far below zero."""
import pytest
import torch

import message_allreduce_amd as llar
from test_gpu_ffn import DTYPES, ids

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
