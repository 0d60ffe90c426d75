"""More rows than one launch has room for: the runtime counts a launch's threads in 32 bits."""
import pytest
import torch

import message_allreduce_amd as llar
from test_gpu_int8 import Draw8, quantized64, same

pytestmark = pytest.mark.gpu


def tall(rows, k, dtype, seed=1):
    """rows x k values, different in every row."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(rows, k, dtype=dtype, device="cuda").normal_(generator=g)


@pytest.mark.parametrize("dtype,rows,k", [(torch.bfloat16, (1 << 26) + 70, 16), (torch.float16, (1 << 27) + 5, 3)], ids=str)
def test_quantize_tall(dtype, rows, k):
    x = tall(rows, k, dtype)
    q, scale = llar.quantize_rows(x)
    for at in (0, (1 << 26) - 40, rows - 3000):
        part = slice(at, min(at + 3000, rows))
        wq, ws = quantized64(x[part])
        assert same(scale[part], ws) and torch.equal(q[part].double(), wq), at


def test_linear_int8_tall():
    """Values that the call quantises, with weights that it copies in the same launch."""
    rows, k, n = (1 << 26) + 70, 24, 8
    x = tall(rows, k, torch.bfloat16)
    d8 = Draw8(2)
    w, ws = d8(n, k), d8.scales(n, k)
    y = llar.linear_int8(x, w, ws)
    for at in (0, (1 << 26) - 40, rows - 3000):
        part = slice(at, min(at + 3000, rows))
        assert torch.equal(y[part], llar.linear_int8(x[part], w, ws)), at
