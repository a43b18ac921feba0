"""MXFP4: the oracle's hand cases and the calls' refusals (CPU), and the CUDA
path against the oracle (GPU): codes and scales bit for bit, products within
the bound of their FP32 additions."""
import ctypes
import os

import numpy as np
import pytest

from oracle import rq_oracle as orc
from rotated_bit_post_b200 import inputs, rq

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(rq.LIB_PATH):
        from rotated_bit_post_b200 import build
        build.build()
    return rq.lib()


# ------------------------------------------------------------------ CPU: oracle
def _block(*head):
    b = np.zeros((1, 32), np.float32)
    b[0, :len(head)] = head
    return b


@pytest.mark.parametrize("head,byte,codes", [
    ((6.0, -3.0, 0.25, 0.75, 1.25), 127, (7, 13, 0, 2, 2)),        # 4 <= amax < 8: scale 1; ties to even
    ((7.9, 4.0, 5.0, 2.5, 3.5), 127, (7, 6, 6, 4, 6)),             # 7.9 saturates at 6
    ((1.0, 0.5, 0.0625, 0.0624), 125, (6, 4, 0, 0)),               # scale 1/4: 4, 2, 0.25 (tie), below
    ((8.0, 1.0, -1.5), 128, (6, 1, 10)),                           # scale 2: 4, 0.5, -0.75 (tie to 1.0)
    ((0.0,), 0, (0,)),                                             # an empty block
    ((2.0 ** -126, 2.0 ** -127), 0, (4, 2)),                       # 2 and 1 on the grid: the exponent stops at 2^-127
    ((3.0e38, 1.0), 252, (7, 0)),
])
def test_oracle_hand_blocks(head, byte, codes):
    q, s = orc.quant_mxfp4(_block(*head))
    assert s[0, 0] == byte
    assert tuple(q[0, :len(codes)]) == codes


def test_oracle_non_finite_block_is_nan_and_alone():
    y = np.ones((2, 64), np.float32)
    y[0, 3], y[1, 40] = np.nan, -np.inf
    q, s = orc.quant_mxfp4(y)
    assert s.tolist() == [[255, 125], [125, 255]]
    assert not q[0, :32].any() and not q[1, 32:].any()
    v = orc.dequant_mxfp4(q, s)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all()


def test_oracle_error_is_half_a_step():
    # nearest grid point: at most half the widest step (2) below 6, and what
    # saturation cuts (8 - 6) above, in units of the block scale
    y = np.random.default_rng(0).standard_normal((64, 256)).astype(np.float32)
    q, s = orc.quant_mxfp4(y)
    err = np.abs(orc.dequant_mxfp4(q, s) - y) / np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)
    inside = np.abs(y) <= 6 * np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)
    assert err[inside].max() <= 1.0 and err.max() <= 2.0


def test_oracle_route_ties_and_nan():
    lg = np.array([[1.0, 3.0, 3.0, 2.0], [np.nan, -1.0, np.nan, -2.0], [np.nan] * 4])
    idx, w = orc.route_top_k(lg, 2, True)
    assert idx.tolist() == [[1, 2], [1, 3], [0, 1]]
    assert np.allclose(w[0], 0.5) and np.isnan(w[2]).all()


# ---------------------------------------------------------------- CPU: refusals
P = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1008)


def test_activation_refusals(L):
    act = lambda K=256, block=64, U=None, r=0, bs=P, codes=P: L.rq_rotate_quantize_act(  # noqa: E731
        rq.MXFP4, P, 0, K, block, P, None, U, r, P if U else None, codes, None, bs, None, None)
    assert act() == 0                          # no row scales: `scale` may be NULL
    assert act(K=192) == 0                     # odd multiples of 64
    assert act(K=160, block=32) == 1 and "multiple of 64" in rq.rq_last_error()
    assert act(bs=None) == 1 and "MXFP4 needs block_scale" in rq.rq_last_error()
    assert act(codes=None) == 1
    assert act(bs=ODD) == 3
    assert act(block=48) == 2 and act(block=2048) == 2
    assert act(K=384, block=128, U=P, r=32) == 0
    assert act(K=384, block=128, U=P, r=12) == 2


def test_product_refusals(L):
    lin = lambda a=rq.MXFP4, w=rq.MXFP4, M=0, N=5, K=192, abs_=P, wbs=P, Y=P: L.rq_w4a4_linear(  # noqa: E731
        a, w, M, N, K, P, None, abs_, P, None, wbs, None, None, None, None, 0, Y, 0, None, None)
    assert lin() == 0
    assert lin(w=rq.NVFP4) == 2 and lin(a=rq.NVFP4) == 2
    assert lin(K=96) == 1 and lin(N=0) == 1 and lin(M=-1) == 1
    assert lin(abs_=None) == 1 and lin(wbs=None) == 1 and "block scales" in rq.rq_last_error()
    assert lin(Y=ODD) == 3


def test_dequantize_refusals(L):
    deq = lambda rows=0, K=64, c=P, s=P, o=P: L.rq_mxfp4_dequantize(rows, K, c, s, o, 0, None)  # noqa: E731
    assert deq() == 0 and deq(c=None, o=None) == 0      # an empty batch
    assert deq(rows=-1) == 1 and deq(K=32) == 1 and deq(K=0) == 1
    assert deq(2, c=None) == 1 and deq(2, s=None) == 1 and deq(2, o=None) == 1
    assert deq(2, o=ODD) == 3


def test_layer_refusals(L):
    ws = rq.rq_mxfp4_layer_workspace(3, 5, 192)
    assert ws >= 3 * 96 + 2 * 512
    assert rq.rq_mxfp4_layer_workspace(3, 5, 100) == -1 and rq.rq_mxfp4_layer_workspace(-1, 5, 128) == -1
    lay = lambda M=0, N=5, K=192, block=64, X=P, rot=P, w=P, s=P, wsp=P, n=1 << 30, Y=P: L.rq_mxfp4_layer(  # noqa: E731
        M, N, K, block, X, rot, w, s, wsp, n, Y, 0, None, None)
    assert lay() == 0 and lay(X=None, Y=None, wsp=None) == 0      # an empty batch
    assert lay(M=3, n=ws - 1) == 1 and "workspace" in rq.rq_last_error()
    assert lay(K=100) == 1 and lay(N=0) == 1 and lay(M=-1) == 1 and lay(block=128) == 1 and lay(block=8) == 2
    for kw in ({"X": None}, {"rot": None}, {"w": None}, {"s": None}, {"wsp": None}, {"Y": None}):
        assert lay(M=3, **kw) == 1, kw
    for kw in ({"X": ODD}, {"rot": ODD}, {"w": ODD}, {"s": ODD}, {"wsp": ODD}, {"Y": ODD}):
        assert lay(M=3, **kw) == 3, kw


def test_moe_refusals(L):
    def moe(T=0, K=192, I=128, E=4, k=2, block=64, block2=64, ptr=None, at=None, n=1 << 40):
        p = [P] * 11
        if at is not None:
            p[at] = ptr
        X, rt, rot, w1, s1, w2, s2, ix, wt, ws, Y = p
        return L.rq_mxfp4_moe(T, K, I, E, k, 1, X, rt, block, rot, w1, s1, block2, w2, s2, ix, wt, ws, n, Y, 0,
                              None, None)
    assert moe() == 0 and moe(at=0) == 0      # an empty batch
    assert moe(T=-1) == 1 and moe(T=65) == 2 and moe(E=257) == 2 and moe(E=0) == 1
    assert moe(k=5) == 1 and moe(k=0) == 1 and moe(E=32, k=17) == 1
    assert moe(K=200) == 1 and moe(I=192) == 1 and moe(block=128) == 1
    assert moe(block=8) == 2 and moe(block2=256) == 2 and moe(block2=24) == 2
    assert moe(T=1, n=rq.rq_mxfp4_moe_workspace(1, 192, 128, 4, 2) - 1) == 1 and "workspace" in rq.rq_last_error()
    for at in range(11):
        assert moe(T=1, at=at, ptr=None) == 1, at
        assert moe(T=1, at=at, ptr=ODD) == 3, at
    assert rq.rq_mxfp4_moe_workspace(65, 192, 128, 4, 2) == -1


def test_binding_checks_sizes(L):
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="block_scale"):
        rq.rq_mxfp4_dequantize(c, s[:100], torch.zeros(4, 64), 1)
    with pytest.raises(ValueError, match="out"):
        rq.rq_mxfp4_dequantize(c, s, torch.zeros(4, 60), 1)
    with pytest.raises(ValueError, match="out"):
        rq.rq_mxfp4_dequantize(c, s, torch.zeros(4, 64), 0)
    with pytest.raises(ValueError, match="device buffer"):
        rq.rq_mxfp4_dequantize(c, s, torch.zeros(4, 64), 1)


def test_binding_refuses_another_device(monkeypatch):
    monkeypatch.setattr(rq, "_current_device", lambda: 0)

    class Far:                        # a tensor of another GPU, as far as the check looks
        def get_device(self):
            return 3
    with pytest.raises(ValueError, match="tensor on device 3"):
        rq._devs(Far())


# ------------------------------------------------------------------ GPU helpers
def _rows(M, K, seed=0):
    rng = np.random.default_rng((seed, M, K))
    x = rng.standard_normal((M, K), dtype=np.float32)
    x[:, rng.choice(K, 3, replace=False)] *= 30
    return inputs.bf16_bits(x * np.exp(0.5 * rng.standard_normal((M, 1))).astype(np.float32))


def _cuda(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _ok(status):
    rc, code = rq.rq_read_status(status)
    assert rc == 0, hex(code)


def _scales(buf, rows, K):
    m, kb = np.arange(rows)[:, None], np.arange(K // 32)[None, :]
    off = (m // 128 * ((K + 127) // 128) + kb // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + kb % 4
    return buf.cpu().numpy()[off]


def _quantize(bits, block, rot_t, U_t=None, rot2_t=None, weight=False):
    """-> codes, scale buffer, coefficients; every byte past the rows' own is checked to be untouched."""
    rows, K = bits.shape
    codes = torch.full(((rows + 2) * (K // 2),), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((rq.mx_sf_bytes(rows, K),), 0xA5, dtype=torch.uint8, device="cuda")
    st = _status()
    coef = None if U_t is None else torch.empty((rows, U_t.shape[1]), dtype=torch.int16, device="cuda")
    X = _cuda(bits)
    view = codes[: rows * (K // 2)].view(rows, K // 2)
    if rot2_t is not None:
        f = rq.rq_quantize_weights2 if weight else rq.rq_rotate_quantize_act2
        f(rq.MXFP4, X, block, rot_t, rot2_t, None, view, None, *((sf, None) if weight else (None, sf)), st)
    else:
        f = rq.rq_quantize_weights if weight else rq.rq_rotate_quantize_act
        f(rq.MXFP4, X, block, rot_t, None, U_t, coef, view, None, sf, st)
    _ok(st)
    assert (codes[rows * (K // 2):] == 0xA5).all()
    pad = np.ones(sf.numel(), bool)
    m, kb = np.arange(rows)[:, None], np.arange(K // 32)[None, :]
    pad[(m // 128 * ((K + 127) // 128) + kb // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + kb % 4] = False
    assert (sf.cpu().numpy()[pad] == 0xA5).all()
    return view, sf, coef


def _assert_codes(view, sf, o, K):
    assert np.array_equal(_scales(sf, view.shape[0], K), o["block_scale"])
    bad = np.argwhere(view.cpu().numpy() != o["codes"])
    assert bad.size == 0, (len(bad), bad[:5].tolist())


def _sum_bound(A, B):
    """FP32 additions of K exact products, a truncating adder allowed: K 2^-23 sum |a b|."""
    return A.shape[1] * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T) + 1e-37


def _packed(values):
    """FP32 rows -> device codes, scale buffer and FP64 values (the oracle's quantizer)."""
    q, s = orc.quant_mxfp4(values)
    rows, K = q.shape
    buf = np.full(rq.mx_sf_bytes(rows, K), 0xFF, np.uint8)     # padding NaN: it must not matter
    m, kb = np.arange(rows)[:, None], np.arange(K // 32)[None, :]
    buf[(m // 128 * ((K + 127) // 128) + kb // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + kb % 4] = s
    return (torch.from_numpy(orc.pack_nibbles(q)).cuda(), torch.from_numpy(buf).cuda(), orc.dequant_mxfp4(q, s))


# ------------------------------------------------------------------ GPU: quantizer
@pytest.mark.gpu
@pytest.mark.parametrize("M,K,block", [(1, 64, 64), (1, 4096, 128), (3, 192, 16), (5, 320, 32), (130, 1152, 128),
                                       (33, 1344, 64), (17, 2048, 256), (9, 1536, 512), (7, 3072, 1024),
                                       (2, 16384, 128), (300, 12288, 256), (1000, 1536, 128), (4, 16384, 1024),
                                       (129, 128, 16), (20000, 128, 32), (9001, 192, 64), (3000, 1536, 128),
                                       (5000, 512, 512), (2500, 4096, 1024), (1300, 16384, 256), (700, 5120, 1024)])
def test_quantize_parity(L, M, K, block):
    bits = _rows(M, K)
    bits[M // 2, : K // 2] = 0
    sign, perm, rot = rq.rq_make_rotation(K, block, 0)
    o = orc.rotate_quantize(inputs.bf16_to_f32(bits), orc.MXFP4, block, sign, perm)
    rot_t = torch.from_numpy(rot).cuda()
    for weight in (False, True):
        view, sf, _ = _quantize(bits, block, rot_t, weight=weight)
        _assert_codes(view, sf, o, K)


@pytest.mark.gpu
def test_quantize_zero_rows_and_extremes(L):
    # rows of zeros, of the smallest and the largest BF16 magnitudes, and of one spike
    K, block = 256, 64
    x = np.zeros((6, K), np.float32)
    x[1], x[2], x[3, 77], x[4, ::2], x[5, 200] = 2.0 ** -126, 2.0 ** 120, 1.0, -3.0, 2.0 ** -120
    bits = inputs.bf16_bits(x)
    sign, perm, rot = rq.rq_make_rotation(K, block, 3)
    o = orc.rotate_quantize(inputs.bf16_to_f32(bits), orc.MXFP4, block, sign, perm)
    view, sf, _ = _quantize(bits, block, torch.from_numpy(rot).cuda())
    _assert_codes(view, sf, o, K)


@pytest.mark.gpu
def test_quantize_non_finite(L):
    # a NaN or infinity spoils its own Hadamard block's scales, nothing else
    K, block, M = 512, 128, 3
    bits = _rows(M, K)
    sign, perm, rot = rq.rq_make_rotation(K, block, 1)
    rot_t = torch.from_numpy(rot).cuda()
    clean, sfc, _ = _quantize(bits, block, rot_t)
    bits[1, 5], bits[2, 9] = 0x7FC0, 0xFF80     # NaN, -infinity
    view, sf, _ = _quantize(bits, block, rot_t)
    s, sc = _scales(sf, M, K), _scales(sfc, M, K)
    for row, ch in ((1, 5), (2, 9)):
        b = int(np.argwhere(perm == ch)[0, 0]) // block
        hit = np.zeros(K // 32, bool)
        hit[b * block // 32: (b + 1) * block // 32] = True
        assert (s[row, hit] == 255).all() and np.array_equal(s[row, ~hit], sc[row, ~hit])
        per = np.repeat(hit, 16)
        c = view.cpu().numpy()[row]
        assert not c[per].any() and np.array_equal(c[~per], clean.cpu().numpy()[row][~per])
    assert np.array_equal(s[0], sc[0])


@pytest.mark.gpu
@pytest.mark.parametrize("K,block,r", [(384, 128, 32), (1152, 128, 8), (1024, 256, 16), (1024, 512, 24)])
def test_quantize_with_low_rank_branch(L, K, block, r):
    bits = _rows(37, K)
    sign, perm, rot = rq.rq_make_rotation(K, block, 0)
    U = np.linalg.qr(np.random.default_rng(5).standard_normal((K, r)))[0].astype(np.float32)
    U_bits = inputs.bf16_bits(U)
    for weight in (False, True):
        o = orc.rotate_quantize(inputs.bf16_to_f32(bits), orc.MXFP4, block, sign, perm, None,
                                inputs.bf16_to_f32(U_bits), weight_rows=weight)
        view, sf, coef = _quantize(bits, block, torch.from_numpy(rot).cuda(), U_t=_cuda(U_bits), weight=weight)
        _assert_codes(view, sf, o, K)
        assert np.array_equal(coef.cpu().numpy().view(np.uint16), o["coef"])


@pytest.mark.gpu
@pytest.mark.parametrize("K,block", [(256, 16), (1152, 128), (2048, 512)])
def test_quantize_double_rotation(L, K, block):
    bits = _rows(35, K)
    sign, perm, _ = rq.rq_make_rotation(K, block, 0)
    ident = np.arange(K, dtype=np.int32)
    rot = np.where(sign < 0, ident | np.int32(-2 ** 31), ident).astype(np.int32)
    mag = np.abs(np.random.default_rng(1).standard_normal(K)).astype(np.float32)
    zz, rot2 = rq.rq_make_zigzag(mag, block)
    o = orc.rotate_quantize(inputs.bf16_to_f32(bits), orc.MXFP4, block, sign, ident, zz_perm=zz)
    for weight in (False, True):
        view, sf, _ = _quantize(bits, block, torch.from_numpy(rot).cuda(), rot2_t=torch.from_numpy(rot2).cuda(),
                                weight=weight)
        _assert_codes(view, sf, o, K)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,K", [(1, 64), (129, 192), (77, 1152)])
def test_dequantize(L, rows, K):
    v = np.random.default_rng(rows).standard_normal((rows, K)).astype(np.float32)
    v[0, :32] = 0
    v[-1, -32:] = np.inf
    codes, sf, ref = _packed(v)
    for fp32, dt in ((1, torch.float32), (0, torch.bfloat16)):
        out = torch.empty((rows, K), dtype=dt, device="cuda")
        rq.rq_mxfp4_dequantize(codes, sf, out, fp32)
        assert np.array_equal(out.double().cpu().numpy(), ref, equal_nan=True)   # every value is exact in BF16
        # an output that is 16-byte aligned and no more, with its neighbours untouched
        n, off = rows * K, 16 // out.element_size()
        wide = torch.full((n + 2 * off,), 7.0, dtype=dt, device="cuda")
        rq.rq_mxfp4_dequantize(codes, sf, wide[off: off + n], fp32)
        assert np.array_equal(wide[off: off + n].view(rows, K).double().cpu().numpy(), ref, equal_nan=True)
        assert (wide[:off] == 7).all() and (wide[off + n:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,block", [(2, 200, 512, 128), (30, 136, 512, 128), (150, 264, 512, 128)])
def test_layer_on_16_byte_aligned_buffers(L, M, N, K, block):
    # every buffer 16 bytes into its allocation: the alignment that the calls ask for, and no more
    X, rot_t, wc, wsf, A, B = _layer_case(M, N, K, block)

    def shifted(t):
        off = 16 // t.element_size()
        s = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")[off:]
        return s.copy_(t.reshape(-1)).view(t.shape)
    ws, st = shifted(_workspace(rq.rq_mxfp4_layer_workspace(M, N, K))), _status()
    for dt in (torch.float32, torch.bfloat16):
        Y = shifted(torch.zeros((M, N), dtype=dt, device="cuda"))
        rq.rq_mxfp4_layer(shifted(X), block, shifted(rot_t), shifted(wc), shifted(wsf), ws, Y, int(dt == torch.float32), st)
        _ok(st)
        # FP32 sums, then half a step of the output's type
        ref = A @ B.T
        assert (np.abs(Y.double().cpu().numpy() - ref) <= _sum_bound(A, B) * 1.01 +
                (np.abs(ref) + _sum_bound(A, B)) * torch.finfo(dt).eps / 2).all()


@pytest.mark.gpu
def test_moe_on_16_byte_aligned_buffers(L):
    m = Moe(5, 192, 128, 4, 2, True, 64, 32)
    idx, w, Y = m.run()

    def shifted(t):
        off = 16 // t.element_size()
        s = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")[off:]
        return s.copy_(t.reshape(-1)).view(t.shape)
    m.w1, m.w2 = tuple(map(shifted, m.w1)), tuple(map(shifted, m.w2))
    m.router_t, m.rot_t = shifted(_cuda(m.router)), shifted(torch.from_numpy(m.rot).cuda())
    bufs = tuple(map(shifted, m.out()))
    got = m.run(bits=shifted(_cuda(m.bits)), bufs=bufs)
    assert all(torch.equal(a, b) for a, b in zip(got, (idx, w, Y)))


# ------------------------------------------------------------------ GPU: product
SHAPES = [(1, 1, 64), (1, 128, 192), (2, 300, 4096), (7, 129, 1152), (8, 256, 320), (16, 1000, 2048), (17, 4100, 512),
          (33, 64, 1344), (64, 640, 1152), (65, 384, 1024), (128, 256, 256), (130, 1153, 320), (257, 515, 1152),
          (1, 77, 16384), (300, 260, 4160),
          (2600, 2104, 192), (2600, 2101, 448), (5000, 1280, 1152), (20000, 400, 2048),
          (300, 19000, 576)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_parity(L, M, N, K):
    rng = np.random.default_rng((M, N, K))
    a = rng.standard_normal((M, K)).astype(np.float32) * np.exp(rng.standard_normal((M, 1))).astype(np.float32)
    ac, asf, A = _packed(a)
    wc, wsf, B = _packed(rng.standard_normal((N, K)).astype(np.float32) * np.float32(0.02))
    ref, st = A @ B.T, _status()
    Y = torch.full((M * N + 64,), float("nan"), device="cuda")
    rq.rq_w4a4_linear(rq.MXFP4, rq.MXFP4, M, N, K, ac, None, asf, wc, None, wsf, None, None, None, None, Y, 1, st)
    _ok(st)
    assert torch.isnan(Y[M * N:]).all()
    Yg = Y[: M * N].view(M, N)
    assert (np.abs(Yg.double().cpu().numpy() - ref) <= _sum_bound(A, B)).all()
    Yb = torch.full((M * N + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    rq.rq_w4a4_linear(rq.MXFP4, rq.MXFP4, M, N, K, ac, None, asf, wc, None, wsf, None, None, None, None, Yb, 0, st)
    _ok(st)
    assert torch.isnan(Yb[M * N:]).all()
    assert torch.equal(Yb[: M * N].view(M, N), Yg.to(torch.bfloat16))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(5, 70, 512), (130, 258, 256)])
def test_product_wide_scales_and_nan_rows(L, M, N, K):
    # scale bytes over their whole useful range; a NaN block spoils its own row
    # (activations) or column (weights) of Y and nothing else
    rng = np.random.default_rng(M)
    a = (rng.standard_normal((M, K)) * np.exp2(rng.integers(-50, 50, (M, 1)))).astype(np.float32)
    b = (rng.standard_normal((N, K)) * np.exp2(rng.integers(-60, 10, (N, 1)))).astype(np.float32)
    a[0] = 0
    a[M // 2, 40] = np.nan
    b[N - 1, 3] = np.inf
    ac, asf, A = _packed(a)
    wc, wsf, B = _packed(b)
    Y, st = torch.empty((M, N), device="cuda"), _status()
    rq.rq_w4a4_linear(rq.MXFP4, rq.MXFP4, M, N, K, ac, None, asf, wc, None, wsf, None, None, None, None, Y, 1, st)
    _ok(st)
    y = Y.double().cpu().numpy()
    bad = np.zeros((M, N), bool)
    bad[M // 2], bad[:, N - 1] = True, True
    assert np.isnan(y[bad]).all()
    A, B = np.nan_to_num(A), np.nan_to_num(B)
    assert (np.abs(y - A @ B.T) <= _sum_bound(A, B))[~bad].all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r", [(3, 100, 256, 8), (64, 132, 192, 16), (200, 300, 1152, 32)])
def test_product_with_low_rank_branch(L, M, N, K, r):
    rng = np.random.default_rng((M, r))
    ac, asf, A = _packed(rng.standard_normal((M, K)).astype(np.float32))
    wc, wsf, B = _packed(rng.standard_normal((N, K)).astype(np.float32) * np.float32(0.02))
    c, l = (inputs.bf16_bits(rng.standard_normal((n, r)).astype(np.float32)) for n in (M, N))
    C, Lr = inputs.bf16_to_f32(c).astype(np.float64), inputs.bf16_to_f32(l).astype(np.float64)
    Y, st = torch.empty((M, N), device="cuda"), _status()
    rq.rq_w4a4_linear(rq.MXFP4, rq.MXFP4, M, N, K, ac, None, asf, wc, None, wsf, None, None, _cuda(c), _cuda(l), Y, 1, st)
    _ok(st)
    ref = A @ B.T + C @ Lr.T
    bound = _sum_bound(np.hstack([A, C]), np.hstack([B, Lr]))
    assert (np.abs(Y.double().cpu().numpy() - ref) <= bound).all()


# -------------------------------------------------------------------- GPU: layer
def _layer_case(M, N, K, block, seed=0):
    bits = _rows(M, K, seed)
    sign, perm, rot = rq.rq_make_rotation(K, block, seed)
    o = orc.rotate_quantize(inputs.bf16_to_f32(bits), orc.MXFP4, block, sign, perm)
    A = orc.dequant_mxfp4(o["q"], o["block_scale"])
    w = np.random.default_rng((seed, N)).standard_normal((N, K)).astype(np.float32) * np.float32(0.02)
    wc, wsf, B = _packed(w)
    return _cuda(bits), torch.from_numpy(rot).cuda(), wc, wsf, A, B


def _workspace(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,block", [(1, 256, 64, 64), (1, 515, 4096, 128), (3, 100, 192, 16), (8, 1000, 1344, 32),
                                         (16, 384, 2048, 1024), (17, 129, 1152, 128), (40, 300, 512, 512),
                                         (64, 256, 8192, 256), (65, 256, 256, 64), (200, 640, 1152, 128),
                                         (2, 64, 16384, 512), (4, 300, 4096, 1024), (2, 640, 8192, 512),
                                         (1, 2305, 1024, 32), (3, 2048, 1344, 64), (1, 129, 8192, 1024),
                                         (4, 4300, 256, 16), (1, 18900, 512, 256), (2, 4200, 1088, 64),
                                         (2, 9473, 8192, 1024), (1, 9600, 6144, 1024)])
def test_layer(L, M, N, K, block):
    X, rot_t, wc, wsf, A, B = _layer_case(M, N, K, block)
    ws, st = _workspace(rq.rq_mxfp4_layer_workspace(M, N, K)), _status()
    Y = torch.full((M * N + 64,), float("nan"), device="cuda")
    rq.rq_mxfp4_layer(X, block, rot_t, wc, wsf, ws, Y, 1, st)
    _ok(st)
    assert torch.isnan(Y[M * N:]).all()
    Yg = Y[: M * N].view(M, N)
    assert (np.abs(Yg.double().cpu().numpy() - A @ B.T) <= _sum_bound(A, B)).all()
    Yb = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    rq.rq_mxfp4_layer(X, block, rot_t, wc, wsf, ws, Yb, 0, st)
    _ok(st)
    assert torch.equal(Yb, Yg.to(torch.bfloat16))   # the same sums in the same order


@pytest.mark.gpu
def test_layer_empty_batch(L):
    X, rot_t, wc, wsf, _, _ = _layer_case(1, 64, 128, 64)
    Y, st = torch.full((4,), 7.0, device="cuda"), _status()
    rq.rq_mxfp4_layer(X[:0], 64, rot_t, wc, wsf, _workspace(256), Y, 1, st)
    _ok(st)
    assert (Y == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 200])
def test_layer_streams_and_graph(L, M):
    # two streams at once, each with its own workspace, then a captured call
    # replayed on new rows: the results of the plain call, bit for bit
    N, K, block = 384, 1024, 128
    X, rot_t, wc, wsf, _, _ = _layer_case(M, N, K, block)
    X2 = _cuda(_rows(M, K, 9))
    st = _status()
    n = rq.rq_mxfp4_layer_workspace(M, N, K)

    def plain(x):
        Y = torch.empty((M, N), device="cuda")
        rq.rq_mxfp4_layer(x, block, rot_t, wc, wsf, _workspace(n), Y, 1, st)
        _ok(st)
        return Y
    want, want2 = plain(X), plain(X2)
    streams, ys, wss = [torch.cuda.Stream() for _ in range(2)], [], [_workspace(n), _workspace(n)]
    torch.cuda.synchronize()
    for rep in range(20):
        for s, x, w in zip(streams, (X, X2), wss):
            with torch.cuda.stream(s):
                Y = torch.empty((M, N), device="cuda")
                rq.rq_mxfp4_layer(x, block, rot_t, wc, wsf, w, Y, 1, st, stream=s)
                ys.append(Y)
    torch.cuda.synchronize()
    _ok(st)
    for i, Y in enumerate(ys):
        assert torch.equal(Y, (want, want2)[i % 2])
    xs, Y, ws = X.clone(), torch.empty((M, N), device="cuda"), _workspace(n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rq.rq_mxfp4_layer(xs, block, rot_t, wc, wsf, ws, Y, 1, st)
    for x, w in ((X, want), (X2, want2), (X, want)):
        xs.copy_(x)
        Y.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, w)


# ---------------------------------------------------------------------- GPU: moe
class Moe:
    """Inputs of a layer and its values in FP64, expert by expert."""

    def __init__(self, T, K, I, E, k, renorm, block, block2, seed=0):
        self.dims = (T, K, I, E, k)
        self.renorm, self.block, self.block2 = renorm, block, block2
        rng = np.random.default_rng((seed, T, K, I, E))
        self.bits = inputs.bf16_bits(rng.standard_normal((T, K)).astype(np.float32))
        self.router = inputs.bf16_bits(rng.standard_normal((E, K)).astype(np.float32) / np.float32(np.sqrt(K)))
        self.sign, self.perm, self.rot = rq.rq_make_rotation(K, block, seed)
        w1 = [_packed(rng.standard_normal((2 * I, K)).astype(np.float32) * np.float32(0.05)) for _ in range(E)]
        w2 = [_packed(rng.standard_normal((K, I)).astype(np.float32) * np.float32(0.05)) for _ in range(E)]
        self.w1_min = min(float(orc_min) for orc_min in (w[1][w[1] != 255].min() for w in w1))
        self.W1, self.W2 = [w[2] for w in w1], [w[2] for w in w2]
        self.w1 = torch.stack([w[0] for w in w1]), torch.stack([w[1] for w in w1])
        self.w2 = torch.stack([w[0] for w in w2]), torch.stack([w[1] for w in w2])

    def out(self, fp32=True):
        T, K, I, E, k = self.dims
        return (torch.full((T, k), -1, dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda"),
                _workspace(rq.rq_mxfp4_moe_workspace(T, K, I, E, k)),
                torch.full((T, K), float("nan"), dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda"))

    def run(self, fp32=True, bits=None, bufs=None, st=None, stream=None):
        idx, w, ws, Y = bufs or self.out(fp32)
        s = st if st is not None else _status()
        x = bits if bits is not None else _cuda(self.bits)
        rq.rq_mxfp4_moe(x, _cuda(self.router) if not hasattr(self, "router_t") else self.router_t, self.dims[4],
                        self.renorm, self.block, torch.from_numpy(self.rot).cuda() if not hasattr(self, "rot_t") else
                        self.rot_t, *self.w1, self.block2, *self.w2, idx, w, ws, Y, int(fp32), s, stream)
        if st is None:
            _ok(s)
        return idx, w, Y

    def reference(self, idx, wts):
        """Y in FP64 for the given experts and weights, and per value how far roundings can move it.

        The products' sums are exact in FP32 in any order (asserted: every partial sum is an integer below
        2^24 in units of the smallest product).  The hidden values then carry at most 8 roundings of 2^-23
        (exp within 2 ulp, a sum, a division, two products) and the transform log2(block2) <= 7 of 2^-24 of
        its partial sums, all below 2^-17 sqrt(block2) max|h|: a value that close to a border of the grid may
        fall on either side of it.  The last sum has at most I k non-zero terms."""
        T, K, I, E, k = self.dims
        x = inputs.bf16_to_f32(self.bits)
        o = orc.rotate_quantize(x, orc.MXFP4, self.block, self.sign, self.perm)
        A = orc.dequant_mxfp4(o["q"], o["block_scale"])
        unit = 2.0 ** (float(o["block_scale"].min()) - 127 + self.w1_min - 127 - 2)
        Y, far = np.zeros((T, K)), np.zeros((T, K))
        H = np.array([[(-1) ** bin(r & c).count("1") for c in range(self.block2)] for r in range(self.block2)])
        for t in range(T):
            for j, e in enumerate(idx[t]):
                assert (np.abs(self.W1[e]) @ np.abs(A[t])).max() < 2.0 ** 24 * unit
                gu = self.W1[e] @ A[t]
                g, u = gu[:I], gu[I:]
                b = (wts[t, j] * g / (1 + np.exp(-g)) * u).reshape(-1, self.block2)
                y = (b @ H / np.sqrt(self.block2)).reshape(1, I)
                d = 2.0 ** -17 * np.repeat(np.abs(b).max(1) * np.sqrt(self.block2), self.block2)[None]
                q0, qp, qm = (orc.dequant_mxfp4(*orc.quant_mxfp4(v.astype(np.float32))) for v in (y, y + d, y - d))
                slack = (np.abs(qp - q0) + np.abs(qm - q0))[0]
                w2 = np.abs(self.W2[e])
                Y[t] += self.W2[e] @ q0[0]
                far[t] += w2 @ slack + I * k * 2.0 ** -23 * (w2 @ (np.abs(q0[0]) + slack))
        return Y, far + 1e-37


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,I,E,k,renorm,block,block2", [
    (1, 64, 128, 1, 1, True, 64, 16), (1, 512, 256, 8, 2, True, 128, 128), (2, 192, 128, 5, 5, False, 16, 32),
    (7, 320, 384, 16, 4, False, 64, 64), (16, 512, 128, 8, 2, True, 512, 128), (33, 1152, 256, 4, 1, True, 128, 128),
    (64, 256, 256, 32, 6, False, 32, 64), (64, 1024, 128, 3, 3, True, 1024, 128), (9, 256, 128, 256, 16, True, 256, 32),
    (1, 2048, 1024, 8, 8, True, 128, 128)])
def test_moe(L, T, K, I, E, k, renorm, block, block2):
    m = Moe(T, K, I, E, k, renorm, block, block2)
    idx, w, Y = m.run()
    gi, gw = idx.cpu().numpy(), w.double().cpu().numpy()
    # the choice: the FP32 sums of K products are off by at most `near`
    x, r = (inputs.bf16_to_f32(b).astype(np.float64) for b in (m.bits, m.router))
    logits, near = x @ r.T, K * 2.0 ** -23 * (np.abs(x) @ np.abs(r).T)
    want, _ = orc.route_top_k(logits, k, renorm)
    for t in range(T):
        assert len(set(gi[t])) == k and gi[t].min() >= 0 and gi[t].max() < E
        for j in np.flatnonzero(gi[t] != want[t]):
            assert abs(logits[t, gi[t, j]] - logits[t, want[t, j]]) <= 2 * near[t].max()
    # the weights: two logits' error in the exponents of numerator and denominator, then FP32
    # roundings of an exponential (2 ulp), a sum of up to E terms and a division
    p = np.exp(logits - logits.max(1, keepdims=True))
    sel = np.take_along_axis(p, gi.astype(np.int64), 1)
    wts = sel / (sel if renorm else p).sum(1, keepdims=True)
    assert (np.abs(gw - wts) <= (4 * near.max() + (E + 8) * 2.0 ** -23) * wts).all()
    ref, far = m.reference(gi, gw)
    assert (np.abs(Y.double().cpu().numpy() - ref) <= far).all()
    _, _, Yb = m.run(fp32=False)
    assert torch.equal(Yb, Y.to(torch.bfloat16))


@pytest.mark.gpu
def test_moe_ties_take_the_lowest_expert(L):
    m = Moe(3, 128, 128, 8, 3, True, 64, 32)
    r = m.router.copy()
    r[1:] = r[1]
    m.bits[2] = 0                      # all logits equal
    m.router = r
    idx, w, Y = m.run()
    gi, gw = idx.cpu().numpy(), w.cpu().numpy()
    x = inputs.bf16_to_f32(m.bits).astype(np.float64)
    lg = x @ inputs.bf16_to_f32(r).astype(np.float64).T
    for t in range(2):
        assert gi[t].tolist() == ([0, 1, 2] if lg[t, 0] > lg[t, 1] else [1, 2, 3])
    assert gi[2].tolist() == [0, 1, 2] and np.allclose(gw[2], 1 / 3, rtol=2.0 ** -22, atol=0)
    assert (Y[2] == 0).all()


@pytest.mark.gpu
def test_moe_non_finite_tokens_stay_alone(L):
    m = Moe(5, 256, 256, 6, 2, True, 64, 64)
    idx0, w0, Y0 = m.run()
    m.bits[1, 7], m.bits[3, 100] = 0x7FC0, 0x7F80      # NaN, infinity
    idx, w, Y = m.run()
    ok = [0, 2, 4]
    assert torch.equal(Y[ok], Y0[ok]) and torch.equal(idx[ok], idx0[ok]) and torch.equal(w[ok], w0[ok])
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[3]).all()
    gi = idx.cpu().numpy()
    assert all(len(set(row)) == 2 and 0 <= min(row) and max(row) < 6 for row in gi)
    assert gi[1].tolist() == [0, 1]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 24])
def test_moe_streams_and_graph(L, T):
    m = Moe(T, 256, 256, 16, 4, True, 128, 64)
    m.router_t, m.rot_t = _cuda(m.router), torch.from_numpy(m.rot).cuda()
    xs = [_cuda(m.bits), _cuda(inputs.bf16_bits(np.random.default_rng(99).standard_normal((T, 256)).astype(np.float32)))]
    want, st = [m.run(bits=x) for x in xs], _status()
    streams, bufs, got = [torch.cuda.Stream() for _ in xs], [], []
    for _ in range(20):
        bufs.append([m.out() for _ in xs])
    torch.cuda.synchronize()
    for pair in bufs:
        for s, x, b in zip(streams, xs, pair):
            with torch.cuda.stream(s):
                got.append(m.run(bits=x, bufs=b, st=st, stream=s))
    torch.cuda.synchronize()
    _ok(st)
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
    x, b = xs[0].clone(), m.out()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.run(bits=x, bufs=b, st=st)
    for i in (0, 1, 0):
        x.copy_(xs[i])
        for v in b:
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((b[0], b[1], b[3]), want[i]))


@pytest.mark.gpu
def test_quantized_layers_together(L):
    # a block as it is used: a linear layer, the expert layer on its output,
    # a linear layer back, every weight quantized by the library
    T, K, I, E, k = 6, 256, 256, 4, 2
    rng = np.random.default_rng(0)
    st = _status()
    _, _, rot = rq.rq_make_rotation(K, 64, 0)
    rot_t = torch.from_numpy(rot).cuda()
    plain_t = torch.arange(I, dtype=torch.int32, device="cuda")    # no signs, no permutation

    def weights(n, cols, table, block):
        W = _cuda(inputs.bf16_bits(rng.standard_normal((n, cols)).astype(np.float32) / np.float32(np.sqrt(cols))))
        b = rq.weight_buffers(rq.MXFP4, n, cols)
        rq.rq_quantize_weights(rq.MXFP4, W, block, table, None, None, None, b["codes"], None, b["block_scale"], st)
        return W.view(torch.bfloat16).double(), b["codes"], b["block_scale"]
    Wa, ca, sa = weights(K, K, rot_t, 64)
    W1, c1, s1 = weights(E * 2 * I, K, rot_t, 64)
    W2, c2, s2 = weights(E * K, I, plain_t, 128)
    X = _cuda(inputs.bf16_bits(rng.standard_normal((T, K)).astype(np.float32)))
    R = _cuda(inputs.bf16_bits(rng.standard_normal((E, K)).astype(np.float32) / 16))
    h, y, z = (torch.empty((T, K), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    ws = _workspace(max(rq.rq_mxfp4_layer_workspace(T, K, K), rq.rq_mxfp4_moe_workspace(T, K, I, E, k)))
    rq.rq_mxfp4_layer(X, 64, rot_t, ca, sa, ws, h, 0, st)
    rq.rq_mxfp4_moe(h, R, k, True, 64, rot_t, c1.view(E, 2 * I, K // 2), s1, 128, c2.view(E, K, I // 2), s2, idx, w,
                    ws, y, 0, st)
    rq.rq_mxfp4_layer(y, 64, rot_t, ca, sa, ws, z, 0, st)
    _ok(st)
    # the rotations cancel: each step is near the unquantized one.  An E2M1 element is off by at most a
    # step, of 2^-2 on average relative (rms below 0.12 of the block's values), on both operands and,
    # in the expert layer, on the hidden row as well
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(h, X.view(torch.bfloat16).double() @ Wa.T) < 0.25
    g = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            gu = W1[e * 2 * I:(e + 1) * 2 * I] @ h[t].double()
            g[t] += float(w[t, j]) * (W2[e * K:(e + 1) * K] @ (gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]))
    assert rel(y, g) < 0.5
    assert rel(z, y.double() @ Wa.T) < 0.25


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 64, 200])
def test_layer_wait_runs_out_then_recovers(L, M):
    # the test hook overstates the first copies' bytes: the bounded waits run
    # out, the call reports it, and the next call is right again
    N, K = 300, 1024
    X, rot_t, wc, wsf, A, B = _layer_case(M, N, K, 128)
    ws, st = _workspace(rq.rq_mxfp4_layer_workspace(M, N, K)), _status()
    Y0, Y = (torch.empty((M, N), device="cuda") for _ in range(2))
    rq.rq_mxfp4_layer(X, 128, rot_t, wc, wsf, ws, Y0, 1, st)
    _ok(st)
    rq.rq_set_wait_limit(5_000_000)
    rq.rq_set_fault_injection(16)
    try:
        rq.rq_mxfp4_layer(X, 128, rot_t, wc, wsf, ws, Y, 1, st)
        rc, code = rq.rq_read_status(st)
    finally:
        rq.rq_set_fault_injection(0)
        rq.rq_set_wait_limit(0)
    assert rc == 5 and code in {0x101, 0x102, 0x103, 0x104, 0x105}
    st.zero_()
    rq.rq_mxfp4_layer(X, 128, rot_t, wc, wsf, ws, Y, 1, st)
    _ok(st)
    assert torch.equal(Y, Y0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 40])
def test_moe_wait_runs_out_then_recovers(L, T):
    m, st = Moe(T, 256, 256, 8, 2, True, 64, 64), _status()
    _, _, Y0 = m.run()
    rq.rq_set_wait_limit(5_000_000)
    rq.rq_set_fault_injection(16)
    try:
        m.run(st=st)
        rc, code = rq.rq_read_status(st)
    finally:
        rq.rq_set_fault_injection(0)
        rq.rq_set_wait_limit(0)
    assert rc == 5 and code in {0x101, 0x102, 0x103, 0x104, 0x105}
    _, _, Y = m.run()
    assert torch.equal(Y, Y0)
