"""Limits of the MXFP4 calls: their workspace sizes and the calls agree on which
shapes are taken (CPU)."""
import ctypes
import os

import pytest

from rotated_bit_post_b200 import rq


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(rq.LIB_PATH):
        from rotated_bit_post_b200 import build
        build.build()
    return rq.lib()


P = ctypes.c_void_p(0x1000)


@pytest.mark.parametrize("M,N,K", [(0, 5, 64), (3, 5, 16384), (3, 5, 16448), (3, 5, 32768), (3, 5, 96), (3, 0, 64),
                                   (-1, 5, 64), (3, 5, 0), (3, 5, -64), (1, 1, 2 ** 31 - 64)])
def test_layer_workspace_is_refused_where_the_call_is(L, M, N, K):
    # an empty batch of the same N and K is checked without touching a buffer
    rc = L.rq_mxfp4_layer(min(M, 0), N, K, 64, P, P, P, P, P, 1 << 40, P, 0, None, None)
    n = rq.rq_mxfp4_layer_workspace(M, N, K)
    assert (n == -1) == (rc != 0), (n, rc)
    if rc == 0:
        assert n >= M * (K // 2) + (M + 127) // 128 * ((K + 127) // 128) * 512
