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
