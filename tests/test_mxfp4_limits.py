"""Limits of the MXFP4 calls (CPU): their workspace sizes and the calls agree on
which shapes are taken, and the binding refuses weights of another shape."""
import ctypes
import os

import pytest

from rotated_bit_post_b200 import rq

torch = pytest.importorskip("torch")


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


# ------------------------------------------------------------- the binding's shapes
def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _layer(K=128, M=3, N=5, w=None):
    w = _u8(N, K // 2) if w is None else w
    rq.rq_mxfp4_layer(torch.zeros(M, K, dtype=torch.bfloat16), 64, torch.zeros(K, dtype=torch.int32), w,
                      _u8(1 << 16), _u8(1 << 16), torch.zeros(1 << 12, dtype=torch.bfloat16), 0,
                      torch.zeros(1, dtype=torch.int32))


def _moe(T=2, K=128, I=128, E=4, k=2, **kw):
    a = {"router": torch.zeros(E, K, dtype=torch.bfloat16), "w1": _u8(E, 2 * I, K // 2), "w2": _u8(E, K, I // 2)}
    a.update(kw)
    rq.rq_mxfp4_moe(torch.zeros(T, K, dtype=torch.bfloat16), a["router"], k, 1, 64, torch.zeros(K, dtype=torch.int32),
                    a["w1"], _u8(1 << 16), 64, a["w2"], _u8(1 << 16), torch.zeros(T, k, dtype=torch.int32),
                    torch.zeros(T, k), _u8(1 << 16), torch.zeros(T, K, dtype=torch.bfloat16), 0,
                    torch.zeros(1, dtype=torch.int32))


def test_layer_refuses_weights_of_another_width(L):
    # wider rows hold enough bytes, but would be read at the wrong pitch
    for w in (_u8(5, 128), _u8(5, 96)):
        with pytest.raises(ValueError, match="w_codes"):
            _layer(w=w)
    with pytest.raises(ValueError, match="device buffer"):     # the right width gets as far as the device check
        _layer()


@pytest.mark.parametrize("name,kw", [
    ("router", {"router": torch.zeros(4, 256, dtype=torch.bfloat16)}),
    ("router", {"router": torch.zeros(5, 128, dtype=torch.bfloat16)}),
    ("w1_codes", {"w1": _u8(4, 256, 128)}),
    ("w1_codes", {"w1": _u8(4, 257, 64)}),
    ("w1_codes", {"w1": _u8(4 * 256 * 64)}),
    ("w2_codes", {"w2": _u8(4, 128, 128)}),
    ("w2_codes", {"w2": _u8(4, 256, 64)}),
    ("w2_codes", {"w2": _u8(8, 128, 64)}),
])
def test_expert_layer_refuses_weights_of_another_shape(L, name, kw):
    with pytest.raises(ValueError, match=name):
        _moe(**kw)


def test_expert_layer_takes_flat_weights(L):
    # w2 and the router may come as flat buffers; the device check is what stops these
    for kw in ({}, {"w2": _u8(4 * 128 * 64)}, {"w2": _u8(4 * 128, 64)}, {"router": torch.zeros(4 * 128, dtype=torch.bfloat16)}):
        with pytest.raises(ValueError, match="device buffer"):
            _moe(**kw)


def test_row_scales_are_ignored(L):
    # MXFP4 has none: whatever stands in their place is not looked at
    odd = ctypes.c_void_p(0x1004)
    for scale in (None, P, odd):
        assert L.rq_rotate_quantize_act(rq.MXFP4, P, 0, 128, 64, P, None, None, 0, None, P, scale, P, None, None) == 0
        assert L.rq_quantize_weights(rq.MXFP4, P, 0, 128, 64, P, None, None, 0, None, P, scale, P, None, None) == 0
        assert L.rq_w4a4_linear(rq.MXFP4, rq.MXFP4, 0, 5, 128, P, scale, P, P, scale, P, None, None, None, None, 0, P, 0,
                                None, None) == 0
    assert L.rq_rotate_quantize_act(rq.NVFP4, P, 0, 128, 64, P, None, None, 0, None, P, odd, P, None, None) == 3
    assert L.rq_w4a4_linear(rq.NVFP4, rq.NVFP4, 0, 5, 128, P, odd, P, P, P, P, None, None, None, None, 0, P, 0,
                            None, None) == 3
