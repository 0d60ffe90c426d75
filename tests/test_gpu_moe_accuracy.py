"""The experts' results against binary64 in the 2-norm of every token (moe_reference has the bound and its reasons)."""
import pytest
import torch

from moe_reference import SHARED, WIDE, Layer, allowed, beyond, definition
from test_gpu_ffn import DTYPES, ids

pytestmark = pytest.mark.gpu


def accuracy_case(size, dtype, int8=False):
    layer = Layer(size, dtype, int8)
    y = layer.call()
    want, flips = definition(layer)
    off, most = beyond(y, want, dtype), allowed(layer, want, flips)
    assert (off <= most).all(), "%s: %.3g of the norm, allowed %.3g" % (
        size, (off / want.norm(dim=1)).max().item(), (most / want.norm(dim=1)).max().item())


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("size", [(1, 256, 512, 256, 8, 2), (24, 520, 264, 520, 12, 4), (50, 128, 512, 6200, 6, 2),
                                  (64, 264, 96, 200, 40, 8)], ids=str)
def test_one_rounding_at_the_end(size, dtype):
    """The inner rows keep more digits than the output's type has: the result is as one rounded once."""
    accuracy_case(size, dtype)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("size", SHARED, ids=str)
def test_shared_column_tiles_and_long_rows(size, int8, dtype):
    accuracy_case(size, dtype, int8)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("size", WIDE, ids=str)
def test_widths_of_a_rank(size, int8, dtype):
    accuracy_case(size, dtype, int8)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("m", [1, 40])
def test_inner_values_beyond_binary16(m, int8, dtype):
    """Inner values of 255 x 256 = 65280 and 256 x 512, results of 2^-8 of them: only fp16's own rows end at 65504."""
    layer = Layer((m, 16, 32, 24, 3, 1), dtype, int8)
    layer.x.zero_()
    layer.x[:, 0] = 256 if not int8 else 127
    for name in ("gate", "up", "down"):
        getattr(layer, name).zero_()
    if int8:
        layer.gate[:, 0, 0], layer.up[:, 0, 0], layer.down[:, :, 0] = 1, 1, 127
        layer.gate_scale.fill_(256 / 127), layer.up_scale.fill_(512 / 127), layer.down_scale.fill_(2.0 ** -8 / 127)
    else:
        layer.gate[:, 0, 0], layer.down[:, :, 0] = 1, 2.0 ** -8
        layer.gate[0, 0, 0] = layer.gate[1, 0, 0] = 255 / 256
        layer.up[:, 0, 0], layer.up[0, 0, 0], layer.up[1, 0, 0] = 2, 1, 1
    layer.weights.fill_(1)
    y = layer.call(activation="none")
    e = layer.experts[:, 0].long()
    if int8:
        assert ((y.float() - 512).abs() <= 512 * 2.0 ** -8).all()
    else:
        want = torch.tensor([255.0, 255.0, 512.0], device="cuda")[e]
        if dtype == torch.float16:
            want[e == 2] = float("inf")
        assert torch.equal(y.float(), want[:, None].expand(m, 24))
