"""Cases of the MXFP4 operators: rotate-and-quantize, the quantized linear layer
and the mixture-of-experts layer for a few tokens.

MXFP4 holds blocks of 32 values as E2M1 elements times a power of two (E8M0
byte).  ``run`` computes an operator in plain torch operations in FP32, or,
with ``own`` set, by the library's calls.  The plain transform follows the
library's stated FP32 order (butterflies in ascending stride, one scaling),
so both give the same codes.
"""
import math

import torch

own = False
_rq = None

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's activations of a decoder-width layer: the latency of the call
        {"name": "quantize 1 x 4096", "kind": "quantize", "M": 1, "K": 4096, "block": 128},
        # a ragged batch whose width is an odd multiple of 64
        {"name": "quantize 517 x 1344", "kind": "quantize", "M": 517, "K": 1344, "block": 64},
        # the input of a wide MLP down-projection (4096 image + 512 text tokens)
        {"name": "quantize 4608 x 12288", "kind": "quantize", "M": 4608, "K": 12288, "block": 256},
        # one token through a linear layer: bound by reading the weights
        {"name": "layer 1 x 4096 x 12288", "kind": "layer", "M": 1, "K": 4096, "N": 12288, "block": 128},
        # a small decode batch, with an output width that is no multiple of 8
        {"name": "layer 19 x 8192 x 4100", "kind": "layer", "M": 19, "K": 8192, "N": 4100, "block": 256},
        # the tiny PixArt-width linear
        {"name": "layer 256 x 1152 x 1152", "kind": "layer", "M": 256, "K": 1152, "N": 1152, "block": 128},
        # the PixArt-like MLP fc1
        {"name": "layer 4096 x 1152 x 4608", "kind": "layer", "M": 4096, "K": 1152, "N": 4608, "block": 128},
        # the Wan-like video MLP with two guidance branches: the largest
        {"name": "layer 65520 x 1536 x 8960", "kind": "layer", "M": 65520, "K": 1536, "N": 8960, "block": 128},
        # one token through a layer of many small experts
        {"name": "moe 1 of 64 top 8", "kind": "moe", "T": 1, "K": 2048, "I": 1024, "E": 64, "top_k": 8,
         "renorm": True, "block": 128, "block2": 128},
        # a ragged decode batch, few large experts, an odd multiple of 64 wide
        {"name": "moe 11 of 8 top 2", "kind": "moe", "T": 11, "K": 1344, "I": 3584, "E": 8, "top_k": 2,
         "renorm": False, "block": 64, "block2": 32},
        # the largest batch the layer takes: nearly every expert is read
        {"name": "moe 64 of 128 top 8", "kind": "moe", "T": 64, "K": 2048, "I": 768, "E": 128, "top_k": 8,
         "renorm": True, "block": 128, "block2": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "layer", "layer", "moe"])
    block = rng.choice([16, 32, 64, 128, 256, 512])
    step = max(64, block)
    if kind == "quantize":
        K = step * max(1, round(_log_int(rng, 256, 12288) / step))
        return {"kind": kind, "M": _log_int(rng, 1, max(1, min(16384, 48000000 // K))), "K": K, "block": block}
    if kind == "layer":
        K = step * max(1, round(_log_int(rng, 256, 8192) / step))
        N = _log_int(rng, 64, 12000)
        return {"kind": kind, "M": _log_int(rng, 1, max(1, min(20000, 800000000000 // (K * N)))), "K": K, "N": N,
                "block": block}
    K = step * max(1, round(_log_int(rng, 512, 4096) / step))
    inner = 128 * rng.randint(2, 16)
    E = rng.choice([4, 8, 16, 32, 60, 64, 128])
    E = max(4, min(E, 400000000 // (3 * K * inner)))
    return {"kind": kind, "T": _log_int(rng, 1, 64), "K": K, "I": inner, "E": E,
            "top_k": min(E, rng.choice([1, 2, 4, 6, 8])), "renorm": rng.random() < 0.5, "block": block,
            "block2": rng.choice([16, 32, 64, 128])}


# ----------------------------------------------------------------- plain forms
def _scale_of(amax):
    """E8M0 byte of a block's largest magnitude: its exponent less two, at least 0."""
    return ((amax.contiguous().view(torch.int32) >> 23) - 2).clamp_(min=0)


def _codes_of(v):
    """Sign and index into GRID of the nearest E2M1 value, ties to the even index."""
    a = v.abs()
    code = (a > 0.25).to(torch.int32) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return code + 8 * (v < 0)


def _blocks(y):
    """y [..., K] FP32 -> codes [..., K] and scale bytes [..., K/32]."""
    b = y.reshape(*y.shape[:-1], y.shape[-1] // 32, 32)
    s = _scale_of(b.abs().amax(-1))
    inv = ((254 - s) << 23).view(torch.float32)
    return _codes_of(b * inv.unsqueeze(-1)).reshape(y.shape), s


def _values(codes, s):
    """The FP32 values that codes [..., K] and scale bytes [..., K/32] stand for."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    v = grid[codes].reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32)
    return (v * torch.exp2(s.float() - 127.0).unsqueeze(-1)).reshape(codes.shape)


def _hadamard(y, block):
    """Orthonormal Walsh-Hadamard transform of every `block` values, ascending strides."""
    shape, h = y.shape, 1
    while h < block:
        p = y.reshape(-1, 2, h)
        y = torch.stack((p[:, 0] + p[:, 1], p[:, 0] - p[:, 1]), 1)
        h *= 2
    return y.reshape(shape) * torch.tensor(1.0 / math.sqrt(block), dtype=torch.float32, device=y.device)


def _rotate(x, rot, block):
    perm = (rot & 0x7FFFFFFF).long()
    v = x.float()[:, perm]
    return _hadamard(torch.where(rot < 0, -v, v), block)


def _unpack(codes, tiles):
    """Packed codes [R, K/2] and scale tiles -> FP32 values [R, K]."""
    R, K = codes.shape[0], codes.shape[1] * 2
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(R, K).int()
    kt = (K + 127) // 128
    s = tiles.reshape(-1, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, kt * 4)[:R, : K // 32]
    return _values(c, s.int())


def _experts(codes, tiles, which=None):
    """Values [n, R, K] of the experts `which` (all of them without it)."""
    E, R, half = codes.shape
    t = tiles.reshape(E, -1)
    if which is not None:
        codes, t = codes[which], t[which]
    n, K = codes.shape[0], half * 2
    kt, rt = (K + 127) // 128, (R + 127) // 128
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(n, R, K).int()
    s = t.reshape(n, rt, kt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, rt * 128, kt * 4)[:, :R, : K // 32]
    return _values(c, s.int())


def _swish(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def _plain_moe(s):
    x, E, k = s["X"], s["E"], s["top_k"]
    T = x.shape[0]
    logits = x.float() @ s["router"].float().t()
    e = torch.exp(logits - logits.amax(-1, keepdim=True))
    # the k largest, ties to the lowest expert
    idx = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :k]
    sel = torch.gather(e, 1, idx)
    w = sel / (sel if s["renorm"] else e).sum(-1, keepdim=True)
    xq = _values(*_blocks(_rotate(x, s["rot"], s["block"])))
    inner = s["I"]
    if T * k <= E:   # the chosen experts of every token, one by one
        which = idx.reshape(-1)
        gu = torch.bmm(_experts(s["w1_codes"], s["w1_bscale"], which),
                       xq.repeat_interleave(k, 0).unsqueeze(-1)).squeeze(-1)
        h = w.reshape(-1, 1) * _swish(gu[:, :inner], gu[:, inner:])
        hq = _values(*_blocks(_hadamard(h, s["block2"])))
        y = torch.bmm(_experts(s["w2_codes"], s["w2_bscale"], which), hq.unsqueeze(-1)).reshape(T, k, -1).sum(1)
    else:            # every expert, the unchosen weighted with zero
        gu = torch.matmul(xq, _experts(s["w1_codes"], s["w1_bscale"]).transpose(1, 2))
        we = torch.zeros(T, E, device=x.device).scatter_(1, idx, w)
        h = we.t().unsqueeze(-1) * _swish(gu[..., :inner], gu[..., inner:])
        hq = _values(*_blocks(_hadamard(h, s["block2"])))
        y = torch.bmm(hq, _experts(s["w2_codes"], s["w2_bscale"]).transpose(1, 2)).sum(0)
    return {"y": y.to(torch.bfloat16), "experts": idx.int(), "weights": w}


# -------------------------------------------------------------------- the cases
def _pack(values):
    """FP32 rows [R, K] -> packed MXFP4 codes [R, K/2] and scale tiles, as the library lays them out."""
    R, K = values.shape
    codes, s = _blocks(values)
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).to(torch.uint8)
    rt, kt = (R + 127) // 128, (K + 127) // 128
    full = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8, device=values.device)
    full[:R, : K // 32] = s.to(torch.uint8)
    tiles = full.reshape(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)
    return packed, tiles


def _weights(gen, R, K):
    return _pack(torch.randn(R, K, device="cuda", generator=gen) * 0.02)


def _expert_weights(gen, E, R, K):
    codes = torch.empty(E, R, K // 2, dtype=torch.uint8, device="cuda")
    tiles = torch.empty(E, (R + 127) // 128 * ((K + 127) // 128) * 512, dtype=torch.uint8, device="cuda")
    for e in range(E):
        codes[e], tiles[e] = _weights(gen, R, K)
    return codes, tiles


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    K, M = case["K"], case.get("M", case.get("T"))
    # activations with a few outlier channels and a scale of each token's own
    x = torch.randn(M, K, device="cuda", generator=gen)
    x[:, torch.randperm(K, device="cuda", generator=gen)[:4]] *= 30.0
    x *= torch.exp(0.5 * torch.randn(M, 1, device="cuda", generator=gen))
    if case["kind"] == "moe":   # the input of an expert layer comes normalised
        x *= torch.rsqrt((x * x).mean(-1, keepdim=True))
    perm = torch.randperm(K, device="cuda", generator=gen).int()
    neg = torch.rand(K, device="cuda", generator=gen) < 0.5
    s = {"kind": case["kind"], "block": case["block"], "X": x.to(torch.bfloat16),
         "rot": torch.where(neg, perm | -0x80000000, perm).int(),
         "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    tiles = (M + 127) // 128 * ((K + 127) // 128) * 512
    if case["kind"] == "quantize":
        s["codes"] = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
        s["bscale"] = torch.empty(tiles, dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    elif case["kind"] == "layer":
        s["w_codes"], s["w_bscale"] = _weights(gen, case["N"], K)
        # scratch: the activations' codes and scales, partial sums of a few tokens' rows
        s["workspace"] = torch.empty(M * (K // 2) + tiles + 32 * min(M, 64) * case["N"] + (1 << 20),
                                     dtype=torch.uint8, device="cuda")
        s["Y"] = torch.empty(M, case["N"], dtype=torch.bfloat16, device="cuda")
    else:
        E, inner, k = case["E"], case["I"], case["top_k"]
        s.update(E=E, I=inner, top_k=k, renorm=case["renorm"], block2=case["block2"])
        s["router"] = (torch.randn(E, K, device="cuda", generator=gen) / math.sqrt(K)).to(torch.bfloat16)
        s["w1_codes"], s["w1_bscale"] = _expert_weights(gen, E, 2 * inner, K)
        s["w2_codes"], s["w2_bscale"] = _expert_weights(gen, E, K, inner)
        # scratch: logits, the activations' and hidden rows' codes and scales, partial sums of the output
        hidden = min(E, M * k) * (M * (inner // 2) + inner // 128 * 512)
        s["workspace"] = torch.empty(4 * M * E + M * (K // 2) + tiles + hidden + 32 * M * K + (1 << 20),
                                     dtype=torch.uint8, device="cuda")
        s["idx"] = torch.empty(M, k, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(M, k, dtype=torch.float32, device="cuda")
        s["Y"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    return s


def _library():
    global _rq
    if _rq is None:
        from rotated_bit_post_b200 import rq
        _rq = rq
    return _rq


def run(s):
    kind = s["kind"]
    if own:
        rq = _library()
        if kind == "quantize":
            rq.rq_rotate_quantize_act(rq.MXFP4, s["X"], s["block"], s["rot"], None, None, None, s["codes"], None,
                                      s["bscale"], s["status"])
            rq.rq_mxfp4_dequantize(s["codes"], s["bscale"], s["values"], 0)
            return s["values"]
        if kind == "layer":
            rq.rq_mxfp4_layer(s["X"], s["block"], s["rot"], s["w_codes"], s["w_bscale"], s["workspace"], s["Y"], 0,
                              s["status"])
            return s["Y"]
        rq.rq_mxfp4_moe(s["X"], s["router"], s["top_k"], s["renorm"], s["block"], s["rot"], s["w1_codes"],
                        s["w1_bscale"], s["block2"], s["w2_codes"], s["w2_bscale"], s["idx"], s["w"], s["workspace"],
                        s["Y"], 0, s["status"])
        return {"y": s["Y"], "experts": s["idx"], "weights": s["w"]}
    if kind == "quantize":
        return _values(*_blocks(_rotate(s["X"], s["rot"], s["block"]))).to(torch.bfloat16)
    if kind == "layer":
        xq = _values(*_blocks(_rotate(s["X"], s["rot"], s["block"])))
        return (xq @ _unpack(s["w_codes"], s["w_bscale"]).t()).to(torch.bfloat16)
    return _plain_moe(s)


def work(case):
    K = case["K"]
    if case["kind"] == "quantize":   # rows in, the table, the values out
        M = case["M"]
        return {"bytes": 2 * M * K + 4 * K + 2 * M * K, "flops": M * K * (math.log2(case["block"]) + 2)}
    packed = 0.5 + 1 / 32            # bytes of one MXFP4 value
    if case["kind"] == "layer":
        M, N = case["M"], case["N"]
        return {"bytes": 2 * M * K + 4 * K + N * K * packed + 2 * M * N, "flops": 2 * M * N * K}
    T, E, inner, k = case["T"], case["E"], case["I"], case["top_k"]
    read = E * (1 - (1 - k / E) ** T)   # experts that some token chose, on average
    return {"bytes": 4 * T * K + 4 * K + 2 * E * K + read * 3 * inner * K * packed + 8 * T * k,
            "flops": 2 * T * E * K + 6 * T * k * inner * K}


# ------------------------------------------------------------------ in 64 bits
def _exact_q(y):
    """Nearest MXFP4 values of FP64 rows [..., K]: E2M1 times 2^(floor(log2 max) - 2)."""
    b = y.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    exp = torch.frexp(top)[1].double() - 3   # top = m * 2^e, 0.5 <= m < 1
    scale = torch.where(top > 0, torch.exp2(exp.clamp(min=-127)), torch.ones_like(top))
    a = (b / scale).abs()
    # spacing of the grid: 0.5 below 2, 1 below 4, 2 above; at most 6
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.sign(b) * q * scale).flatten(-2)


def _exact_h(y, block):
    m = torch.ones(1, 1, dtype=torch.float64, device=y.device)
    while m.shape[0] < block:
        m = torch.cat((torch.cat((m, m), 1), torch.cat((m, -m), 1)), 0)
    return (y.unflatten(-1, (-1, block)) @ (m / math.sqrt(block))).flatten(-2)


def _exact_x(s):
    sign = 1.0 - 2.0 * (s["rot"] < 0).double()
    x = s["X"].double().index_select(1, (s["rot"] & 0x7FFFFFFF).long()) * sign
    return _exact_q(_exact_h(x, s["block"]))


def _exact_w(codes, tiles):
    """FP64 values of packed rows, every scale looked up at its place in the tiles."""
    R, half = codes.shape
    grid = torch.tensor(GRID, dtype=torch.float64, device=codes.device)
    c = torch.empty(R, 2 * half, dtype=torch.long, device=codes.device)
    c[:, 0::2] = codes % 16
    c[:, 1::2] = codes // 16
    m = torch.arange(R, device=codes.device).unsqueeze(1)
    kb = torch.arange(half // 16, device=codes.device).unsqueeze(0)
    tk = (2 * half + 127) // 128
    at = (m // 128 * tk + kb // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + kb % 4
    scale = torch.exp2(tiles[at].double() - 127.0).repeat_interleave(32, 1)
    return grid[c % 8] * (1.0 - 2.0 * (c // 8).double()) * scale


def exact(case, seed):
    s = prepare(case, seed)
    xq = _exact_x(s)
    if case["kind"] == "quantize":
        return xq
    if case["kind"] == "layer":
        w, out = _exact_w(s["w_codes"], s["w_bscale"]), torch.empty(s["Y"].shape, dtype=torch.float64, device="cuda")
        for i in range(0, xq.shape[0], 8192):
            torch.mm(xq[i: i + 8192], w.t(), out=out[i: i + 8192])
        return out
    inner, E, k = case["I"], case["E"], case["top_k"]
    p = torch.softmax(s["X"].double() @ s["router"].double().t(), -1)
    w, idx = torch.topk(p, k, dim=-1)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    y = torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel():
            gu = xq[t] @ _exact_w(s["w1_codes"][e], s["w1_bscale"][e]).t()
            g, u = gu[:, :inner], gu[:, inner:]
            h = w[t, j].unsqueeze(1) * g * torch.sigmoid(g) * u
            y.index_add_(0, t, _exact_q(_exact_h(h, case["block2"])) @ _exact_w(s["w2_codes"][e], s["w2_bscale"][e]).t())
    return {"y": y, "experts": idx.int(), "weights": w}
