"""The MXFP4 products when a wait runs out with more steps left than the ring
has stages: the call reports it, nothing faults, and the next call is right.

The test hook overstates the first copies' bytes, so that the first stage's
barrier never completes.  A stage must not be handed back to the copies then:
the next ones would arrive on a barrier whose phase has no arrivals left."""
import os

import numpy as np
import pytest

from rotated_bit_post_b200 import inputs, rq

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(rq.LIB_PATH):
        from rotated_bit_post_b200 import build
        build.build()
    return rq.lib()


class injected:
    """Waits of 5 ms, the first of which run out."""

    def __enter__(self):
        rq.rq_set_wait_limit(5_000_000)
        rq.rq_set_fault_injection(16)

    def __exit__(self, *exc):
        rq.rq_set_fault_injection(0)
        rq.rq_set_wait_limit(0)


TIMEOUT_CODES = {0x101, 0x102, 0x103, 0x104, 0x105}


def _codes(g, *shape):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)


def _scale(g, n):
    return torch.randint(120, 124, (n,), dtype=torch.uint8, device="cuda", generator=g)


def _bf16(rows, K, seed):
    x = np.random.default_rng(seed).standard_normal((rows, K)).astype(np.float32)
    return torch.from_numpy(inputs.bf16_bits(x).view(np.int16)).cuda()


def _runs_out_then_recovers(call, outs, st):
    call()
    assert rq.rq_read_status(st) == (0, 0)
    want = [o.clone() for o in outs]
    for _ in range(2):
        with injected():
            call()
            rc, code = rq.rq_read_status(st)
        assert rc == 5 and code in TIMEOUT_CODES
        st.zero_()
        call()
        assert rq.rq_read_status(st) == (0, 0)
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3, 9600, 8192), (40, 9600, 8192), (64, 256, 32768), (65, 300, 8192),
                                   (300, 520, 4096), (700, 9600, 2048)])
def test_product_of_many_steps(L, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    a, sa, w, sw = _codes(g, M, K // 2), _scale(g, rq.mx_sf_bytes(M, K)), _codes(g, N, K // 2), _scale(g, rq.mx_sf_bytes(N, K))
    Y, st = torch.empty((M, N), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    _runs_out_then_recovers(lambda: rq.rq_w4a4_linear(
        rq.MXFP4, rq.MXFP4, M, N, K, a, None, sa, w, None, sw, None, None, None, None, Y, 1, st), [Y], st)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,block", [(1, 9600, 8192, 128), (3, 9600, 4096, 64), (4, 18900, 2048, 256), (20, 9600, 4096, 128),
                                         (2000, 640, 4096, 128)])
def test_layer_of_many_steps(L, M, N, K, block):
    g = torch.Generator(device="cuda").manual_seed(M)
    _, _, rot = rq.rq_make_rotation(K, block, 0)
    X, rot_t = _bf16(M, K, M), torch.from_numpy(rot).cuda()
    w, sw = _codes(g, N, K // 2), _scale(g, rq.mx_sf_bytes(N, K))
    Y, st = torch.empty((M, N), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(rq.rq_mxfp4_layer_workspace(M, N, K), dtype=torch.uint8, device="cuda")
    _runs_out_then_recovers(lambda: rq.rq_mxfp4_layer(X, block, rot_t, w, sw, ws, Y, 1, st), [Y], st)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,I,E,k", [(20, 4096, 512, 8, 2), (40, 256, 1024, 32, 4), (64, 1024, 2048, 16, 4)])
def test_expert_layer_of_many_steps(L, T, K, I, E, k):
    g = torch.Generator(device="cuda").manual_seed(T)
    _, _, rot = rq.rq_make_rotation(K, 64, 0)
    X, R, rot_t = _bf16(T, K, T), _bf16(E, K, 1), torch.from_numpy(rot).cuda()
    w1, s1 = _codes(g, E, 2 * I, K // 2), _scale(g, E * rq.mx_sf_bytes(2 * I, K))
    w2, s2 = _codes(g, E, K, I // 2), _scale(g, E * rq.mx_sf_bytes(K, I))
    idx, wt = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    Y, st = torch.empty((T, K), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(rq.rq_mxfp4_moe_workspace(T, K, I, E, k), dtype=torch.uint8, device="cuda")
    _runs_out_then_recovers(lambda: rq.rq_mxfp4_moe(
        X, R, k, True, 64, rot_t, w1, s1, 64, w2, s2, idx, wt, ws, Y, 1, st), [Y, idx, wt], st)


# A wait that runs out takes its limit of 5 ms and up to 4 ms of attempts; the bounded wait for the copies
# already issued as long again; the steps still issued, and the launch, are microseconds.  2 x 9 ms, and
# as much again for a machine that is shared.
ENDS_WITHIN_MS = 36.0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 64, 65, 300])
def test_long_product_ends_soon_after_a_wait_runs_out(L, M):
    # 4096 steps of 256 columns, 512 for each of eight ranks in the few-token form: what is left of them
    # when the first wait runs out must not take an attempt each
    N, K = 64, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(M)
    a, sa, w, sw = _codes(g, M, K // 2), _scale(g, rq.mx_sf_bytes(M, K)), _codes(g, N, K // 2), _scale(g, rq.mx_sf_bytes(N, K))
    Y, st = torch.empty((M, N), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    took = []

    def call():
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        rq.rq_w4a4_linear(rq.MXFP4, rq.MXFP4, M, N, K, a, None, sa, w, None, sw, None, None, None, None, Y, 1, st)
        e1.record()
        e1.synchronize()
        took.append(e0.elapsed_time(e1))
    _runs_out_then_recovers(call, [Y], st)
    # normal, expired, normal, expired, normal
    assert all(5.0 <= ms <= ENDS_WITHIN_MS for ms in took[1::2]), took
