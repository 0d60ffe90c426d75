"""Where a row's scale leaves binary32: its largest magnitude over 127 is 0 or the least subnormal number."""
import pytest
import torch

import message_allreduce_amd as llar
from test_gpu_int8 import quantize_case

pytestmark = pytest.mark.gpu


def test_least_scales():
    """63 / 127 of the least number is below its half, 64 / 127 above; there a quotient may pass 127, and is cut."""
    x = torch.zeros(6, 40, device="cuda")
    tops = [0, 1, 63, 64, 190, 191]
    for row, top in enumerate(tops):
        x[row, 3], x[row, 30] = top * 2.0 ** -149, -(top // 3) * 2.0 ** -149
    quantize_case(x)
    q, scale = llar.quantize_rows(x)
    assert (scale.double() * 2.0 ** 149).tolist() == [0, 0, 0, 1, 1, 2]
    assert q[:, 3].tolist() == [0, 0, 0, 64, 127, 96] and q[:, 30].tolist() == [0, 0, 0, -21, -63, -32]
    y = llar.linear_int8(x, torch.full((24, 40), 127, dtype=torch.int8, device="cuda"), torch.full((24,), 2.0 ** 120, device="cuda"))
    assert (y[:3] == 0).all() and (y[3:] > 0).all()
