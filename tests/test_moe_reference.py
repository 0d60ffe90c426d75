"""The comparison of the experts' results finds what it is there to find, at every size that it is used with: outputs of
zeros, a choice or a share of the inner width left out, operands or inner rows with fewer digits.  No GPU: the mistakes
are made in the definition."""
import pytest
import torch

from moe_reference import SHARED, WIDE, Layer, allowed, beyond, definition

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# one token of the wide layers stands for all, and only its own experts are needed
SIZES = SHARED + sorted({(1, k, n, outs, top_k + 1, top_k) for _, k, n, outs, _, top_k in WIDE})


def rejected(layer, y, want, flips):
    return beyond(y.to(layer.dtype), want, layer.dtype) > allowed(layer, want, flips)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_what_is_left_out_is_found(size, int8):
    layer = Layer(size, torch.float32, int8, device="cpu")
    want, flips = definition(layer)
    chosen = layer.experts.clone()
    e = int(chosen[0, 0])
    layer.experts[:, 0] = -1
    choice = definition(layer)[0]
    layer.experts = chosen
    share = {4: 32, 2: 64, 1: 128}  # 128 bytes of an inner row, the least that workgroups share
    for dtype in DTYPES:
        layer.dtype = dtype
        assert not rejected(layer, want, want, flips).any()
        assert rejected(layer, torch.zeros_like(want), want, flips).all()
        assert rejected(layer, choice, want, flips).all()
        width = share[1 if int8 else torch.finfo(dtype).bits // 8]
        last = size[2]
        short = definition(layer, gone=(e, max(last - width, 0), last))[0]
        assert rejected(layer, short, want, flips)[(chosen == e).any(1)].all()


@pytest.mark.parametrize("size", [s for s in SIZES if s[0] * s[3] >= 500 and s[1] * s[2] <= 4096 * 1024], ids=str)
def test_fewer_digits_are_found(size):
    for dtype in (torch.bfloat16, torch.float16):
        layer = Layer(size, dtype, device="cpu")
        want, flips = definition(layer)
        assert rejected(layer, definition(layer, inner=dtype)[0], want, flips).any()
    layer = Layer(size, torch.float32, device="cpu")
    want, flips = definition(layer)
    for name in ("x", "gate", "up", "down"):
        setattr(layer, name, getattr(layer, name).bfloat16().float())
    assert rejected(layer, definition(layer)[0], want, flips).all()
