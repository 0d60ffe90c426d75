"""The tensor-parallel feed-forward layer of examples/tp_feed_forward.py: the
operators and the AllReduce together, against the same layer on one rank in
binary32.

Every tensor between two operators is bfloat16 (relative rounding at most 2^-8,
about 2^-9.8 in the 2-norm): h, the partials, their sum (forward) and dh, dg and
du, dx and its sum (backward).  Six such roundings in a row stay below 2^-7 in
the 2-norm."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("ranks,hidden,inner,tokens", [(8, 1024, 2048, 1), (4, 512, 1000, 37), (2, 264, 520, 300),
                                                       (1, 256, 256, 16), (3, 72, 190, 5)])
def test_layer_matches_one_rank(ranks, hidden, inner, tokens):
    import tp_feed_forward
    status, worst, _ = tp_feed_forward.run(ranks, hidden, inner, tokens)
    assert status == 0
    assert max(worst.values()) < 2.0 ** -7, worst
