// A mixture-of-experts layer on MXFP4 experts, for a few tokens:
//   logits = x Wr^T, the top_k largest per token (ties: the lowest expert),
//   w = their softmax (over the chosen experts, or over all of them),
//   xq = Q(R x), g, u = W1[e] xq, h = w silu(g) u,  hq = Q(H h), y = sum_e W2[e] hq.
// The routing weight goes onto the hidden row before its quantization, so the
// sum over a token's experts is one long contraction.
//
// Three launches, each a programmatic dependent of the one before: routing
// with the activation transform (here), the gate/up products with the hidden
// rows' quantization, the down products with the sum (rq_mxfew.cu).
//
// Routing: a cluster of up to eight CTAs per token.  Every CTA stages the
// token's row, takes its share of the experts' logits (a warp per expert, 16-byte
// reads; FP32 sums) and of the rotated blocks; the logits meet in the
// first CTA's shared memory, where one warp picks the experts.  The split
// keeps one token's pass over the router (E K 2 bytes) off a single SM.  5 us
// for one token and 64 experts, 12 us for 64 tokens and 128 experts (K = 2048).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rq_internal.h"
#include "rq_mx.cuh"
#include "rq_ptx.cuh"

namespace rq {

namespace {

constexpr int PREP_THREADS = 256;
constexpr int MOE_EMAX = 256;

struct PrepParams {
  const uint16_t* x;
  const uint16_t* router;
  const int32_t* rot;
  int32_t* idx;
  float* wts;
  uint8_t *xq, *xq_sf;   // T x K/2 codes, one row tile of scales
  int T, K, E, top_k, renorm, block, cluster;
  float inv_sqrt_b;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A logit as an unsigned key of the same order: -0 as +0, NaN as -infinity,
// never 0 (the key of an expert that is taken or does not exist).
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (l != l) l = -INFINITY;
  const uint32_t b = __float_as_uint(l + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(PREP_THREADS) moe_route_kernel(const __grid_constant__ PrepParams p) {
  extern __shared__ __align__(16) uint16_t xs[];   // the token's row
  __shared__ float logit[MOE_EMAX];
  const int C = p.cluster, rank = (int)blockIdx.x % C, t = blockIdx.x / C;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the gate/up kernel may be scheduled: it waits for this grid before it reads
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int chunks = p.K / 8;   // 16-byte units of a row
  const uint4* xrow = reinterpret_cast<const uint4*>(p.x + (size_t)t * p.K);
  for (int i = threadIdx.x; i < chunks; i += PREP_THREADS) reinterpret_cast<uint4*>(xs)[i] = __ldg(xrow + i);
  __syncthreads();
  // the first CTA's shared memory is written below: all CTAs have started
  cluster_sync();
  uint32_t home;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(home) : "r"(smem_u32(logit)), "r"(0));
  // two experts per warp and turn: twice the reads in flight
  const int stride = C * (PREP_THREADS / 32);
  for (int e = rank + warp * C; e < p.E; e += 2 * stride) {
    const bool two = e + stride < p.E;
    const uint4* w0 = reinterpret_cast<const uint4*>(p.router + (size_t)e * p.K);
    const uint4* w1 = reinterpret_cast<const uint4*>(p.router + (size_t)(two ? e + stride : e) * p.K);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = lane; i < chunks; i += 32) {
      const uint4 a = __ldg(w0 + i), c = __ldg(w1 + i), b = reinterpret_cast<const uint4*>(xs)[i];
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w}, cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        s[0] = fmaf(bf_lo(aw[q]), bf_lo(bw[q]), s[0]);
        s[1] = fmaf(bf_hi(aw[q]), bf_hi(bw[q]), s[1]);
        s[2] = fmaf(bf_lo(cw[q]), bf_lo(bw[q]), s[2]);
        s[3] = fmaf(bf_hi(cw[q]), bf_hi(bw[q]), s[3]);
      }
    }
    s[0] += s[1];
    s[2] += s[3];
#pragma unroll
    for (int m = 16; m; m >>= 1) {
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], m);
      s[2] += __shfl_xor_sync(0xffffffffu, s[2], m);
    }
    if (lane == 0) {
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(home + e * 4), "f"(s[0]) : "memory");
      if (two) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(home + (e + stride) * 4), "f"(s[2]) : "memory");
    }
  }
  // rotated blocks, whole Hadamard blocks per warp and turn
  const int nu = p.K / (p.block < 64 ? 64 : p.block);
  const auto sink = [&](int, int k, uint8_t*& codes, uint8_t*& sf) {
    codes = p.xq + (size_t)t * (p.K / 2) + k / 2;
    sf = p.xq_sf + mx_sf_offset(t, k / 32, p.K);
    return true;
  };
  mx_rotate_units(xs, 0, p.rot, 0, nu, nu, rank + warp * C, C * (PREP_THREADS / 32), p.block,
                  p.inv_sqrt_b, sink);
  cluster_sync();
  if (rank != 0 || warp != 0) return;
  // ------------------------------------------------------------ the top_k experts
  float l[MOE_EMAX / 32];
  uint32_t key[MOE_EMAX / 32];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < MOE_EMAX / 32; ++i) {
    const int e = i * 32 + lane;
    l[i] = e < p.E ? logit[e] : -INFINITY;
    key[i] = e < p.E ? logit_key(l[i]) : 0u;
    mx = fmaxf(mx, l[i]);   // (a NaN is left out)
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < MOE_EMAX / 32; ++i)
    if (i * 32 + lane < p.E) all += expf(l[i] - mx);
#pragma unroll
  for (int m = 16; m; m >>= 1) all += __shfl_xor_sync(0xffffffffu, all, m);
  float sel = 0.f, mine = 0.f;
  int chosen = 0;
  for (int j = 0; j < p.top_k; ++j) {
    uint32_t k = 0u, e = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < MOE_EMAX / 32; ++i)
      if (key[i] > k) { k = key[i]; e = i * 32 + lane; }   // the lowest of this lane's equals
    const uint32_t top = __reduce_max_sync(0xffffffffu, k);
    const uint32_t best = __reduce_min_sync(0xffffffffu, k == top ? e : 0xffffffffu);
#pragma unroll
    for (int i = 0; i < MOE_EMAX / 32; ++i)
      if (best == (uint32_t)(i * 32 + lane)) key[i] = 0u;
    const float ex = expf(logit[best] - mx);
    sel += ex;
    if (lane == j) { mine = ex; chosen = (int)best; }
  }
  if (lane < p.top_k) {
    p.idx[t * p.top_k + lane] = chosen;
    p.wts[t * p.top_k + lane] = __fdiv_rn(mine, p.renorm ? sel : all);
  }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t moe_workspace_bytes(int T, int K, int I, int E, int top_k) {
  const size_t A = E < T * top_k ? E : T * top_k;
  return up256((size_t)T * (K / 2)) + up256(mx_sf_bytes(T, K)) + up256(A * T * (I / 2)) + up256(A * mx_sf_bytes(T, I));
}

cudaError_t launch_moe(const MoeLaunch& a, cudaStream_t st) {
  const int active = a.E < a.T * a.top_k ? a.E : a.T * a.top_k;
  uint8_t* xq = a.ws;
  uint8_t* xq_sf = xq + up256((size_t)a.T * (a.K / 2));
  uint8_t* hq = xq_sf + up256(mx_sf_bytes(a.T, a.K));
  uint8_t* hq_sf = hq + up256((size_t)active * a.T * (a.I / 2));
  PrepParams p{};
  p.x = a.x; p.router = a.router; p.rot = a.rot; p.idx = a.idx; p.wts = a.wts;
  p.xq = xq; p.xq_sf = xq_sf;
  p.T = a.T; p.K = a.K; p.E = a.E; p.top_k = a.top_k; p.renorm = a.renorm; p.block = a.block;
  p.inv_sqrt_b = a.inv_sqrt_b;
  // CTAs per token: eight while they all fit the GPU twice
  p.cluster = 8;
  while (p.cluster > 1 && a.T * p.cluster > 2 * (a.num_sms > 0 ? a.num_sms : 148)) p.cluster /= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.T * p.cluster));
  cfg.blockDim = dim3(PREP_THREADS);
  cfg.dynamicSmemBytes = (size_t)a.K * 2;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, moe_route_kernel, p);
  if (e != cudaSuccess) return e;
  return launch_moe_products(a, xq, xq_sf, hq, hq_sf, active, st);
}

}  // namespace rq
