"""Argument checks of the mixture-of-experts C calls, which need no GPU: a refused call enqueues nothing."""
import ctypes

import pytest

import message_allreduce_amd as llar


@pytest.fixture(scope="module")
def L():
    return llar.lib()


def mat(rows, cols, rs=None, cs=1, data=4096):
    return (ctypes.c_int64 * 5)(data, rows, cols, cols if rs is None else rs, cs)


def experts(e, rows, cols, es=None, rs=None, data=4096):
    rs = cols if rs is None else rs
    return (ctypes.c_int64 * 6)(data, e, rows, cols, rows * rs if es is None else es, rs)


SPACE, BYTES = 4096, 1 << 40  # an address that no refused call touches


def test_route(L):
    def call(x, r, top_k=2, score=0, weights=4096, ids=4096, dtype=2, space=SPACE, n=BYTES):
        return L.llar_moe_route(x, r, top_k, score, 1, weights, ids, dtype, space, n, None)

    ok = (mat(4, 64), mat(8, 64))
    assert call(None, ok[1]) == -1 and call(ok[0], None) == -1
    assert call(*ok, dtype=3) == -1 and call(*ok, score=2) == -1 and call(*ok, top_k=-1) == -1
    assert call(*ok, top_k=9) == -1 and call(*ok, weights=None) == -1 and call(*ok, ids=None) == -1
    assert call(ok[0], mat(8, 63)) == -1
    assert call(mat(4, 64, 1, 4), ok[1]) == -2 and call(ok[0], mat(8, 64, 1, 8)) == -2
    assert call(ok[0], mat(1025, 64)) == -2 and call(ok[0], mat(64, 64), top_k=33) == -2
    wide = (mat(4, 8192), mat(64, 8192))
    assert call(*ok, space=4097) == -1 and call(*wide, n=L.llar_moe_route_workspace(4, 64, 8192) - 1) == -1
    assert call(mat(0, 64), ok[1], weights=None) == 0 and call(*ok, top_k=0, ids=None) == 0  # nothing to do
    assert L.llar_moe_route_workspace(4, 64, 8192) >= 4 * 64 * 8 and L.llar_moe_route_workspace(4, 1024, 0) >= 4 * 1024 * 8
    assert L.llar_moe_route_workspace(4, 8, 64) == 0              # one kernel
    for bad in ((-1, 64, 8192), (4, 1025, 8192), (4, -1, 8192), (4, 64, -1), (4, 64, 1 << 21)):
        assert L.llar_moe_route_workspace(*bad) == 0


def test_ffn(L):
    def call(x, g, u, d, out, ids=4096, id_bytes=4, weights=4096, top_k=2, gs=None, us=None, ds=None, residual=None,
             dtype=2, act=4, space=SPACE, n=BYTES):
        return L.llar_moe_ffn(x, ids, id_bytes, weights, top_k, g, u, d, gs, us, ds, residual, out, dtype, act, space, n,
                              None)

    ok = (mat(4, 64), experts(8, 32, 64), experts(8, 32, 64), experts(8, 64, 32), mat(4, 64))

    def but(i, m):
        return [m if j == i else o for j, o in enumerate(ok)]

    for i in range(5):
        assert call(*but(i, None)) == -1
    assert call(*ok, dtype=3) == -1 and call(*ok, act=7) == -1 and call(*ok, id_bytes=2) == -1 and call(*ok, top_k=-1) == -1
    assert call(*ok, ids=None) == -1 and call(*ok, weights=None) == -1 and call(*ok, top_k=33) == -2
    assert call(*but(0, mat(4, 63))) == -1 and call(*but(0, mat(5, 64))) == -1 and call(*but(0, mat(4, 64, 1, 4))) == -2
    assert call(*but(1, experts(7, 32, 64))) == -1 and call(*but(2, experts(8, 31, 64))) == -1
    assert call(*but(2, experts(8, 32, 64, 5000))) == -2 and call(*but(2, experts(8, 32, 64, 32 * 64, 72))) == -2
    assert call(*but(3, experts(8, 64, 31))) == -1 and call(*but(3, experts(8, 63, 32))) == -1
    assert call(*but(3, experts(8, 64, 32, data=0))) == -1 and call(*but(3, experts(8, 64, 32, -1))) == -1
    assert call(*but(3, experts(-8, 64, 32))) == -1
    many = [mat(4, 64), experts(1025, 32, 64), experts(1025, 32, 64), experts(1025, 64, 32), mat(4, 64)]
    assert call(*many) == -2
    assert call(*but(4, mat(4, 64, 32))) == -1 and call(*but(4, mat(4, 64, 1, 4))) == -2
    assert call(*ok, residual=mat(4, 63)) == -1 and call(*ok, residual=mat(4, 64, 1, 4)) == -2
    for scales in ({"gs": 4096}, {"gs": 4096, "us": 4096}, {"ds": 4096}):  # all three or none
        assert call(*ok, **scales) == -1
    long = [mat(4, 1 << 17), experts(8, 32, 1 << 17), experts(8, 32, 1 << 17), ok[3], ok[4]]
    assert call(*long, gs=4096, us=4096, ds=4096) == -2            # sums that may not fit 32 bits
    def room(m=4, n=32, k=64, outs=64, count=8, top_k=2, dtype=2, int8=0):
        return L.llar_moe_workspace(m, n, k, outs, count, top_k, dtype, int8)

    assert room() >= 4 * 2 * 32 * 2 and call(*ok, n=room() - 1) == -1 and call(*ok, space=4097) == -1
    assert room(int8=1) > room() and room(m=1024, int8=1) == room(m=64, int8=1)
    assert room(m=64, n=4096, outs=48, count=1000, top_k=8) > 64 * 8 * 4096 * 2          # shares of a column tile's experts
    for bad in ({"m": -1}, {"n": -1}, {"k": -1}, {"outs": -1}, {"count": -1}, {"count": 1025}, {"top_k": 33}, {"top_k": -1},
                {"dtype": 3}, {"k": 1 << 21}):
        assert room(**bad, int8=1) == 0
    assert call(*but(0, mat(0, 64))[:4], mat(0, 64), ids=None) == 0  # nothing to do
