// A mixture-of-experts layer on MXFP4 experts, for a few tokens:
//   logits = x Wr^T, the top_k largest per token (ties: the lowest expert),
//   w = their softmax (over the chosen experts, or over all of them),
//   xq = Q(R x), g, u = W1[e] xq, h = w silu(g) u,  hq = Q(H h), y = sum_e W2[e] hq.
// The routing weight goes onto the hidden row before its quantization, so the
// sum over a token's experts is one long contraction.
//
// Three launches: routing with the activation transform, gate/up products
// with the hidden rows' quantization, down products with the sum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rq_internal.h"
#include "rq_mx.cuh"
#include "rq_ptx.cuh"

namespace rq {

namespace {

constexpr int MOE_TMAX = 64;    // tokens
constexpr int MOE_EMAX = 256;   // experts
constexpr int PREP_THREADS = 256;

struct MoeParams {
  const uint16_t* x;
  const uint16_t* router;
  const int32_t* rot;
  const uint8_t *w1, *w1_sf, *w2, *w2_sf;
  int32_t* idx;
  float* wts;
  uint8_t *xq, *xq_sf;   // T x K/2 codes, one row tile of scales
  uint8_t *hq, *hq_sf;   // [active][T][I/2] codes, [active] row tiles of scales
  void* Y;
  int T, K, I, E, top_k, renorm, block, block2, out_fp32;
  float inv_sqrt_b, inv_sqrt_b2;
  int32_t* status;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// ascending list of the experts that some token chose: bits[8] and their count
__device__ __forceinline__ int active_bits(const int32_t* idx, int n, uint32_t* bits) {
  if (threadIdx.x < 8) bits[threadIdx.x] = 0u;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const uint32_t e = (uint32_t)__ldcg(idx + i);
    atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  int c = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) c += __popc(bits[i]);
  return c;
}
// the a-th expert of the list (a < count)
__device__ __forceinline__ int nth_active(const uint32_t* bits, int a) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const int c = __popc(bits[i]);
    if (a < c) return i * 32 + (int)__fns(bits[i], 0, a + 1);
    a -= c;
  }
  return 0;
}

// Butterflies over `n` shared values in blocks of `b`, ascending strides, by the
// whole CTA; ends with a barrier.
__device__ void fwht_shared(float* v, int n, int b) {
  for (int h = 1; h < b; h <<= 1) {
    __syncthreads();
    for (int i = threadIdx.x; i < n / 2; i += blockDim.x) {
      const int lo = (i / h) * 2 * h + i % h;
      const float a = v[lo], c = v[lo + h];
      v[lo] = __fadd_rn(a, c);
      v[lo + h] = __fsub_rn(a, c);
    }
  }
  __syncthreads();
}

// One warp quantizes 32 values (one block): lane l holds value l.
__device__ __forceinline__ void quantize_warp(float y, int m, int kb, int K, uint8_t* codes, uint8_t* sf) {
  const int lane = threadIdx.x & 31;
  float a = fabsf(y);
#pragma unroll
  for (int s = 16; s; s >>= 1) a = fmax_nan(a, __shfl_xor_sync(0xffffffffu, a, s));
  const uint32_t sb = mx_scale_byte(a);
  const float v = __fmul_rn(y, mx_inv_scale(sb));
  const float hi = __shfl_down_sync(0xffffffffu, v, 1);
  if (!(lane & 1)) codes[(size_t)m * (K / 2) + kb * 16 + lane / 2] = sb == 255u ? 0 : cvt_e2m1x2(hi, v);
  if (lane == 0) sf[mx_sf_offset(m, kb, K)] = (uint8_t)sb;
}

// One CTA per token: logits, routing, rotation, quantization.
__global__ void __launch_bounds__(PREP_THREADS) moe_prep_kernel(const MoeParams p) {
  extern __shared__ float sm[];
  float* v = sm;                 // K rotated values
  __shared__ float logit[MOE_EMAX];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint16_t* x = p.x + (size_t)t * p.K;
  for (int i = threadIdx.x; i < p.K; i += blockDim.x) {
    const int32_t r = p.rot[i];
    const float a = bf16_bits_to_f32(x[r & 0x7fffffff]);
    v[i] = r < 0 ? -a : a;
  }
  for (int e = warp; e < p.E; e += PREP_THREADS / 32) {
    const uint16_t* w = p.router + (size_t)e * p.K;
    float s = 0.f;
    for (int i = lane; i < p.K; i += 32) s += bf16_bits_to_f32(w[i]) * bf16_bits_to_f32(x[i]);
    s = warp_sum(s);
    if (lane == 0) logit[e] = s;
  }
  fwht_shared(v, p.K, p.block);
  for (int kb = warp; kb < p.K / 32; kb += PREP_THREADS / 32)
    quantize_warp(__fmul_rn(v[kb * 32 + lane], p.inv_sqrt_b), t, kb, p.K, p.xq, p.xq_sf);
  if (threadIdx.x == 0) {
    float mx = -INFINITY, all = 0.f, sel = 0.f;
    for (int e = 0; e < p.E; ++e) mx = fmaxf(mx, logit[e]);
    for (int e = 0; e < p.E; ++e) all += expf(logit[e] - mx);
    for (int j = 0; j < p.top_k; ++j) {
      int best = -1;
      for (int e = 0; e < p.E; ++e) {   // NaN logits rank as -inf; an expert is chosen once
        bool used = false;
        for (int q = 0; q < j; ++q) used |= p.idx[t * p.top_k + q] == e;
        const float l = logit[e] == logit[e] ? logit[e] : -INFINITY;
        const float b = best >= 0 ? (logit[best] == logit[best] ? logit[best] : -INFINITY) : 0.f;
        if (!used && (best < 0 || l > b)) best = e;
      }
      p.idx[t * p.top_k + j] = best;
      sel += expf(logit[best] - mx);
    }
    for (int j = 0; j < p.top_k; ++j)
      p.wts[t * p.top_k + j] = __fdiv_rn(expf(logit[p.idx[t * p.top_k + j]] - mx), p.renorm ? sel : all);
  }
}

// sum over a row's blocks of scale_w scale_x sum q_w q_x
__device__ float mx_dot(const uint8_t* a, const uint8_t* a_sf, int am, const uint8_t* b, const uint8_t* b_sf, int bm, int K) {
  float s = 0.f;
  for (int kb = 0; kb < K / 32; ++kb) {
    const uint4 qa = *reinterpret_cast<const uint4*>(a + (size_t)am * (K / 2) + kb * 16);
    const uint4 qb = *reinterpret_cast<const uint4*>(b + (size_t)bm * (K / 2) + kb * 16);
    const uint32_t wa[4] = {qa.x, qa.y, qa.z, qa.w}, wb[4] = {qb.x, qb.y, qb.z, qb.w};
    float d = 0.f;
    for (int i = 0; i < 4; ++i)
      for (int e = 0; e < 8; ++e) d += e2m1_value(wa[i] >> (4 * e) & 15u) * e2m1_value(wb[i] >> (4 * e) & 15u);
    s += d * mx_scale(a_sf[mx_sf_offset(am, kb, K)]) * mx_scale(b_sf[mx_sf_offset(bm, kb, K)]);
  }
  return s;
}

// CTA (active expert, 128 hidden channels): gate and up rows, hidden row, quantization.
__global__ void __launch_bounds__(256) moe_gate_up_kernel(const MoeParams p) {
  __shared__ uint32_t bits[8];
  __shared__ float gu[256];
  __shared__ float wt;
  __shared__ int routed;
  const int n = active_bits(p.idx, p.T * p.top_k, bits);
  const int a = blockIdx.x, c0 = blockIdx.y * 128;
  if (a >= n) return;
  const int e = nth_active(bits, a);
  const uint8_t* w1 = p.w1 + (size_t)e * 2 * p.I * (p.K / 2);
  const uint8_t* s1 = p.w1_sf + (size_t)e * mx_sf_bytes(2 * p.I, p.K);
  uint8_t* hq = p.hq + (size_t)a * p.T * (p.I / 2);
  uint8_t* hs = p.hq_sf + (size_t)a * mx_sf_bytes(p.T, p.I);
  const int c = threadIdx.x & 127;
  const int row = (threadIdx.x < 128 ? 0 : p.I) + c0 + c;
  for (int t = 0; t < p.T; ++t) {
    if (threadIdx.x == 0) {
      routed = 0;
      for (int j = 0; j < p.top_k; ++j)
        if (p.idx[t * p.top_k + j] == e) {
          wt = p.wts[t * p.top_k + j];
          routed = 1;
        }
    }
    __syncthreads();
    const float w = wt;
    const bool on = routed != 0;
    if (on) gu[threadIdx.x] = mx_dot(w1, s1, row, p.xq, p.xq_sf, t, p.K);
    __syncthreads();
    if (on && threadIdx.x < 128) {
      const float g = gu[c], u = gu[c + 128];
      gu[c] = __fmul_rn(w, __fmul_rn(__fdiv_rn(g, __fadd_rn(1.f, expf(-g))), u));
    } else if (threadIdx.x < 128) {
      gu[c] = 0.f;
    }
    fwht_shared(gu, 128, p.block2);
    if (threadIdx.x < 128)
      quantize_warp(__fmul_rn(gu[c], p.inv_sqrt_b2), t, (c0 + c) / 32, p.I, hq, hs);
    __syncthreads();
  }
}

// CTA (128 output channels, token): the sum over the active experts, in order.
__global__ void __launch_bounds__(128) moe_down_kernel(const MoeParams p) {
  __shared__ uint32_t bits[8];
  const int n = active_bits(p.idx, p.T * p.top_k, bits);
  const int row = blockIdx.x * 128 + threadIdx.x, t = blockIdx.y;
  if (row >= p.K) return;
  float s = 0.f;
  for (int a = 0; a < n; ++a) {
    const int e = nth_active(bits, a);
    bool on = false;
    for (int j = 0; j < p.top_k; ++j) on |= p.idx[t * p.top_k + j] == e;
    if (on)
      s += mx_dot(p.w2 + (size_t)e * p.K * (p.I / 2), p.w2_sf + (size_t)e * mx_sf_bytes(p.K, p.I), row,
                  p.hq + (size_t)a * p.T * (p.I / 2), p.hq_sf + (size_t)a * mx_sf_bytes(p.T, p.I), t, p.I);
  }
  if (p.out_fp32) static_cast<float*>(p.Y)[(size_t)t * p.K + row] = s;
  else static_cast<__nv_bfloat16*>(p.Y)[(size_t)t * p.K + row] = __float2bfloat16_rn(s);
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t moe_workspace_bytes(int T, int K, int I, int E, int top_k) {
  const size_t A = E < T * top_k ? E : T * top_k;
  return up256((size_t)T * (K / 2)) + up256(mx_sf_bytes(T, K)) + up256(A * T * (I / 2)) + up256(A * mx_sf_bytes(T, I));
}

cudaError_t launch_moe(const MoeLaunch& a, cudaStream_t st) {
  MoeParams p{};
  p.x = a.x; p.router = a.router; p.rot = a.rot;
  p.w1 = a.w1; p.w1_sf = a.w1_sf; p.w2 = a.w2; p.w2_sf = a.w2_sf;
  p.idx = a.idx; p.wts = a.wts; p.Y = a.Y;
  p.T = a.T; p.K = a.K; p.I = a.I; p.E = a.E; p.top_k = a.top_k; p.renorm = a.renorm;
  p.block = a.block; p.block2 = a.block2; p.out_fp32 = a.out_fp32;
  p.inv_sqrt_b = a.inv_sqrt_b; p.inv_sqrt_b2 = a.inv_sqrt_b2;
  p.status = a.status;
  const int A = a.E < a.T * a.top_k ? a.E : a.T * a.top_k;
  uint8_t* ws = a.ws;
  p.xq = ws;
  p.xq_sf = p.xq + up256((size_t)a.T * (a.K / 2));
  p.hq = p.xq_sf + up256(mx_sf_bytes(a.T, a.K));
  p.hq_sf = p.hq + up256((size_t)A * a.T * (a.I / 2));
  const int smem = a.K * 4;
  cudaError_t e = cudaFuncSetAttribute(moe_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  moe_prep_kernel<<<a.T, PREP_THREADS, smem, st>>>(p);
  moe_gate_up_kernel<<<dim3(A, a.I / 128), 256, 0, st>>>(p);
  moe_down_kernel<<<dim3((a.K + 127) / 128, a.T), 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace rq
