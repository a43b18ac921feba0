"""MXFP4 corners on the GPU: ranks of a cluster that no step falls to, the
low-rank branch with BF16 output, and expert layers of more than 2048 channels."""
import numpy as np
import pytest

from rotated_bit_post_b200 import inputs, rq
from tests import test_mxfp4 as mx

torch = pytest.importorskip("torch")
L = mx.L      # the module's fixture: the built library


def one_expert(T, K, I, E, which):
    """Every token's best expert is `which`: a large first channel that its router row alone reads."""
    m = mx.Moe(T, K, I, E, 1, True, 64, 64)
    x, r = inputs.bf16_to_f32(m.bits).copy(), inputs.bf16_to_f32(m.router).copy()
    x[:, 0], r[:, 0] = 4.0, 0.0
    r[which, 0] = 16.0
    m.bits, m.router = inputs.bf16_bits(x), inputs.bf16_bits(r)
    return m


def check(m):
    idx, w, Y = m.run()
    ref, far = m.reference(idx.cpu().numpy(), w.double().cpu().numpy())
    assert (np.abs(Y.double().cpu().numpy() - ref) <= far).all()
    _, _, Yb = m.run(fp32=False)
    assert torch.equal(Yb, Y.to(torch.bfloat16))
    return idx, w


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,I,E,which", [(16, 256, 128, 8, 3), (40, 192, 256, 64, 63), (64, 1152, 128, 32, 0)])
def test_all_tokens_on_one_expert(L, T, K, I, E, which):
    # the down products are split for min(E, T) experts, of which one is chosen: a step or
    # two for up to eight ranks, the others add zeros
    idx, w = check(one_expert(T, K, I, E, which))
    assert (idx == which).all() and (w == 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,I,E,k", [(5, 2112, 128, 3, 2), (3, 4160, 256, 4, 2), (2, 128, 4224, 4, 3), (7, 2304, 2432, 2, 1)])
def test_wide_expert_layers(L, T, K, I, E, k):
    check(mx.Moe(T, K, I, E, k, True, 64, 128))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r", [(1, 132, 192, 32), (64, 300, 320, 24), (65, 129, 256, 8), (200, 300, 1152, 32),
                                     (1, 132, 8192, 32), (4, 101, 4096, 8), (8, 520, 8192, 16), (64, 260, 16384, 16)])
def test_low_rank_product_in_bf16(L, M, N, K, r):
    rng = np.random.default_rng((M, r))
    ac, asf, A = mx._packed(rng.standard_normal((M, K)).astype(np.float32))
    wc, wsf, B = mx._packed(rng.standard_normal((N, K)).astype(np.float32) * np.float32(0.02))
    c, l = (inputs.bf16_bits(rng.standard_normal((n, r)).astype(np.float32)) for n in (M, N))
    A, B = np.hstack([A, inputs.bf16_to_f32(c)]), np.hstack([B, inputs.bf16_to_f32(l)])
    Y, st = torch.full((M * N + 64,), float("nan"), dtype=torch.bfloat16, device="cuda"), mx._status()
    rq.rq_w4a4_linear(rq.MXFP4, rq.MXFP4, M, N, K, ac, None, asf, wc, None, wsf, None, None, mx._cuda(c), mx._cuda(l), Y, 0, st)
    mx._ok(st)
    assert torch.isnan(Y[M * N:]).all()
    # the FP32 sums, then half a step of BF16
    ref, near = A @ B.T, mx._sum_bound(A, B)
    y = Y[: M * N].view(M, N).double().cpu().numpy()
    assert (np.abs(y - ref) <= near + (np.abs(ref) + near) * 2.0 ** -8).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r", [(64, 12288, 4096, 32), (64, 4608, 1152, 32), (16, 1152, 1152, 16)])
def test_low_rank_branch_has_no_cliff(L, M, N, K, r):
    # up to 64 tokens a product may take the few-token kernel, whose low-rank branch costs r per token in
    # the epilogue; one token more never does.  The same work within a factor of three (it was 12 to 14).
    g = torch.Generator(device="cuda").manual_seed(0)
    w, sw = (torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda", generator=g) for n in (N * K // 2, rq.mx_sf_bytes(N, K)))
    Lr, st = torch.zeros((N, r), dtype=torch.int16, device="cuda"), mx._status()

    def us(m):
        a, sa = torch.zeros((m, K // 2), dtype=torch.uint8, device="cuda"), torch.zeros(rq.mx_sf_bytes(m, K), dtype=torch.uint8, device="cuda")
        c, Y = torch.zeros((m, r), dtype=torch.int16, device="cuda"), torch.empty((m, N), dtype=torch.bfloat16, device="cuda")
        call = lambda: rq.rq_w4a4_linear(rq.MXFP4, rq.MXFP4, m, N, K, a, None, sa, w.view(N, K // 2), None, sw, None, None, c, Lr, Y, 0, st)  # noqa: E731
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(10):
                call()
        took = []
        for _ in range(9):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            graph.replay()
            e1.record()
            e1.synchronize()
            took.append(e0.elapsed_time(e1) * 100)
        return sorted(took)[4]
    few, more = us(M), us(65)
    mx._ok(st)
    assert few < 3 * more, (few, more)
