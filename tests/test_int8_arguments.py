"""Argument checks of the 8-bit products' C calls, which need no GPU: a refused call enqueues nothing."""
import ctypes

import pytest

import message_allreduce_amd as llar


@pytest.fixture(scope="module")
def L():
    return llar.lib()


def mat(rows, cols, rs=None, cs=1, data=4096):
    return (ctypes.c_int64 * 5)(data, rows, cols, cols if rs is None else rs, cs)


SPACE, BYTES = 4096, 1 << 40  # an address that no refused call touches


def test_quantize_rows(L):
    def call(x, q, scale=4096, dtype=2):
        return L.llar_quantize_rows(x, q, scale, dtype, None)

    ok = (mat(4, 64), mat(4, 64))
    assert call(None, ok[1]) == -1 and call(ok[0], None) == -1 and L.llar_last_error() == -1
    assert call(*ok, dtype=3) == -1 and call(*ok, scale=None) == -1
    assert call(ok[0], mat(4, 63)) == -1 and call(ok[0], mat(3, 64)) == -1
    assert call(ok[0], mat(4, 64, 32)) == -1                       # output rows overlap
    assert call(ok[0], mat(4, 64, 1, 4)) == -2                     # output columns not contiguous
    assert call(mat(4, 64, data=0), ok[1]) == -1 and call(mat(4, 64, -64), ok[1]) == -1
    assert call(mat(4, (1 << 30) + 8), mat(4, (1 << 30) + 8)) == -2
    assert call(mat(4, 1 << 21), mat(4, 1 << 21)) == -2            # longest contiguous axis: 2^21 - 8
    assert call(mat(0, 64), mat(0, 64), scale=None) == 0           # nothing to do


def test_linear_int8(L):
    def call(x, w, out, xs=4096, ws=4096, dtype=2, act=0, residual=None, space=SPACE, n=BYTES):
        return L.llar_linear_int8(x, xs, w, ws, None, residual, out, dtype, act, space, n, None)

    ok = (mat(4, 64), mat(32, 64), mat(4, 32))
    for i in range(3):
        assert call(*[None if j == i else m for j, m in enumerate(ok)]) == -1
    assert call(*ok, dtype=7) == -1 and call(*ok, act=9) == -1 and call(*ok, act=-1) == -1 and call(*ok, ws=None) == -1
    assert call(mat(4, 63), *ok[1:]) == -1 and call(*ok[:2], mat(4, 31)) == -1 and call(*ok[:2], mat(5, 32)) == -1
    assert call(mat(4, 64, 1, 4), *ok[1:]) == -2                   # whole numbers: contiguous rows
    assert call(ok[0], mat(32, 64, 1, 32), ok[2]) == -2
    assert call(*ok[:2], mat(4, 32, 1, 4)) == -2 and call(*ok[:2], mat(4, 32, 16)) == -1
    assert call(*ok, residual=mat(4, 32, 1, 4)) == -2 and call(*ok, residual=mat(4, 31)) == -1
    assert call(mat(4, 1 << 17), mat(32, 1 << 17), ok[2]) == -2    # sums that may not fit 32 bits
    assert call(mat(4, 64, -64), *ok[1:]) == -1 and call(mat(-1, 64), *ok[1:]) == -1
    assert call(*ok, space=4096 + 8) == -1                         # misaligned workspace
    # no room for the whole numbers
    assert call(*ok, xs=None, n=0) == -1 and call(mat(1, 64, 1, 8), ok[1], mat(1, 32), xs=None, n=0) == -1
    assert call(mat(0, 64), mat(32, 64), mat(0, 32)) == 0 and call(mat(4, 64), mat(0, 64), mat(4, 0), ws=None) == 0


def test_gated_ffn_int8(L):
    def call(x, g, u, out, gs=4096, us=4096, dtype=2, act=4, space=SPACE, n=BYTES):
        return L.llar_gated_ffn_int8(x, 4096, g, u, gs, us, out, dtype, act, space, n, None)

    ok = (mat(4, 64), mat(32, 64), mat(32, 64), mat(4, 32))
    for i in range(4):
        assert call(*[None if j == i else m for j, m in enumerate(ok)]) == -1
    assert call(*ok, gs=None) == -1 and call(*ok, us=None) == -1 and call(*ok, dtype=5) == -1 and call(*ok, act=5) == -1
    assert call(ok[0], ok[1], mat(31, 64), ok[3]) == -1 and call(ok[0], ok[1], mat(32, 64, 80), ok[3]) == -2
    assert call(ok[0], ok[1], mat(32, 64, 1, 32), ok[3]) == -2
    assert call(mat(4, 1 << 17), mat(32, 1 << 17), mat(32, 1 << 17), ok[3]) == -2


def test_workspace(L):
    def need(m, n, k, layout, op=0):
        return L.llar_int8_workspace(op, m, n, k, layout)

    assert need(1, 512, 512, 0) == 0 and need(4, 512, 512, 16) >= 4 * 512 + 16 and need(1, 512, 512, 18) >= 512 + 4
    assert need(100, 512, 512, 1) >= need(100, 512, 512, 0) + 512 * 512
    assert need(100, 512, 512, 1, 2) >= need(100, 512, 512, 0, 2) + 2 * 512 * 512
    for bad in ((-1, 8, 8), (8, -1, 8), (8, 8, -1), (8, 8, 1 << 17), ((1 << 30) + 1, 8, 8)):
        assert need(*bad, 17) == 0
    assert need(8, 8, 8, 17, 1) == 0 and need(8, 8, 8, 17, 3) == 0  # no such operators
    for dims in ((0, 8, 8), (3, 0, 8), (3, 8, 0), (0, 0, 0)):
        for layout in (0, 1, 16, 17):
            assert need(*dims, layout) < 4096
