"""Sizes that the experts' kernels have no room for are refused before anything is enqueued.  No GPU needed."""
import message_allreduce_amd as llar
from test_moe_arguments import BYTES, SPACE, experts, mat


def call(m, n, k, outs, count, top_k):
    return llar.lib().llar_moe_ffn(mat(m, k), 4096, 4, 4096, top_k, experts(count, n, k), experts(count, n, k),
                                   experts(count, outs, n), None, None, None, None, mat(m, outs), 2, 4, SPACE, BYTES, None)


def test_too_many_workgroups():
    assert call(64, 1 << 17, 8, 8, 1024, 16) == -2                # 2^13 column tiles of 1024 experts
    assert call(32, 1 << 18, 8, 8, 1024, 16) == -2                # of 512 choices
    assert call(1, 8, 8, 1 << 27, 4, 2) == -2                     # outputs, 16 a workgroup
    assert call(70, 8, 8, (1 << 28) - 8, 4, 2) == -2 and call(69, 8, 8, 1 << 28, 4, 2) == -2
    assert call(64, 8, 8, 1 << 28, 4, 2) == -2                    # 32 a workgroup
