// MXFP4 pieces shared by the kernels: blocks of 32 values held as E2M1
// elements times a power of two, 2^(byte - 127) (E8M0; OCP Microscaling
// specification), scale bytes in 128-row x 128-column tiles of 512 bytes.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "rq_ptx.cuh"

namespace rq {

// Scale byte (m, kb), kb = k / 32: tile (m / 128, kb / 4), inside it
// (m%32)*16 + ((m%128)/32)*4 + kb%4, the 32 x 16-byte form tcgen05.cp moves.
__host__ __device__ __forceinline__ size_t mx_sf_offset(int m, int kb, int K) {
  const int tiles_k = (K + 127) / 128;
  return ((size_t)(m >> 7) * tiles_k + (kb >> 2)) * 512 + (m & 31) * 16 + ((m >> 5) & 3) * 4 + (kb & 3);
}
__host__ __device__ __forceinline__ size_t mx_sf_bytes(int rows, int K) {
  return (size_t)((rows + 127) / 128) * ((K + 127) / 128) * 512;
}

// max that keeps a NaN operand, so that a block holding one shows it
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale byte of a block from its largest magnitude: floor(log2 amax) - 2 (the
// largest E2M1 exponent), not below 2^-127; 255 (NaN) when amax is not finite.
// Zero and subnormal maxima take byte 0.
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
  const uint32_t e = (__float_as_uint(amax) >> 23) & 0xFFu;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - byte), the factor that brings the block onto the E2M1 grid; 0 for
// byte 255 (its elements are stored as zeros).
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127); NaN for byte 255.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}
// E2M1 nibble -> value
__device__ __forceinline__ float e2m1_value(uint32_t n) {
  const uint32_t m = n & 7u;
  const float a = m < 2u ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  return n & 8u ? -a : a;
}

// One warp transforms and quantizes 32 EPL rotated coordinates from `base` on, EPL
// consecutive ones per lane, of the BF16 row xs (shared memory), row number m:
// butterflies in ascending stride, inside the lane and then across lanes.  rot: the
// table's entries from `base` on.  sink(m, k, codes, sf) says where coordinate k's
// packed codes and its block's scale byte go, or false for nowhere.
template <int EPL, class Sink>
__device__ __forceinline__ void mx_rotate_epl(const uint16_t* xs, int m, const int32_t* rot, int base, int block, float isb,
                                              const Sink& sink) {
  const int lane = threadIdx.x & 31, k0 = base + lane * EPL;
  float v[EPL];
  int32_t tab[EPL];
  if constexpr (EPL >= 4) {
#pragma unroll
    for (int i = 0; i < EPL; i += 4)
      *reinterpret_cast<int4*>(tab + i) = *reinterpret_cast<const int4*>(rot + lane * EPL + i);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) tab[i] = rot[lane * EPL + i];
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int32_t r = tab[i];
    v[i] = __uint_as_float(((uint32_t)xs[r & 0x7fffffff] << 16) ^ ((uint32_t)r & 0x80000000u));
  }
#pragma unroll
  for (int h = 1; h < EPL; h <<= 1) {   // (EPL <= block)
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (!(i & h)) {
        const float a = v[i], b = v[i + h];
        v[i] = __fadd_rn(a, b);
        v[i + h] = __fsub_rn(a, b);
      }
  }
  for (int s = 1; s * EPL < block; s <<= 1) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, v[i], s);
      v[i] = lane & s ? __fsub_rn(o, v[i]) : __fadd_rn(v[i], o);
    }
  }
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    v[i] = __fmul_rn(v[i], isb);
    am = fmax_nan(am, fabsf(v[i]));
  }
#pragma unroll
  for (int s = 1; s < 32 / EPL; s <<= 1) am = fmax_nan(am, __shfl_xor_sync(0xffffffffu, am, s));
  const uint32_t sb = mx_scale_byte(am);
  const float inv = mx_inv_scale(sb);
  uint8_t *dst, *sf;
  if (!sink(m, k0, dst, sf)) return;
  uint32_t w[(EPL + 7) / 8];
#pragma unroll
  for (int i = 0; i < (EPL + 7) / 8; ++i) w[i] = 0u;
#pragma unroll
  for (int i = 0; i < EPL; i += 2)
    w[i / 8] |= (sb == 255u ? 0u : (uint32_t)cvt_e2m1x2(__fmul_rn(v[i + 1], inv), __fmul_rn(v[i], inv))) << (4 * (i & 7));
  if constexpr (EPL == 2) *dst = (uint8_t)w[0];
  else if constexpr (EPL == 4) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w[0];
  else if constexpr (EPL == 8) *reinterpret_cast<uint32_t*>(dst) = w[0];
  else if constexpr (EPL == 16) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  if (k0 % 32 == 0) *sf = (uint8_t)sb;
}
// Units of max(block, 64) coordinates, whole Hadamard blocks: unit j of `all` is
// coordinates (u0 + j % nu) U ... of row j / nu; this warp takes j = first, first +
// stride, ..., two at a time so that one's latencies cover the other's.  rot: the
// table's entries from u0 U on.
template <int EPL, class Sink>
__device__ __forceinline__ void mx_rotate_loop(const uint16_t* rows, int K, const int32_t* rot, int u0, int nu, int all,
                                               int first, int stride, int block, float isb, const Sink& sink) {
#pragma unroll 2
  for (int j = first; j < all; j += stride) {
    const int m = j / nu, u = j - m * nu;
    mx_rotate_epl<EPL>(rows + (size_t)m * K, m, rot + u * 32 * EPL, (u0 + u) * 32 * EPL, block, isb, sink);
  }
}
template <class Sink>
__device__ __forceinline__ void mx_rotate_units(const uint16_t* rows, int K, const int32_t* rot, int u0, int nu, int all,
                                                int first, int stride, int block, float isb, const Sink& sink) {
  if (block <= 64) mx_rotate_loop<2>(rows, K, rot, u0, nu, all, first, stride, block, isb, sink);
  else if (block == 128) mx_rotate_loop<4>(rows, K, rot, u0, nu, all, first, stride, 128, isb, sink);
  else if (block == 256) mx_rotate_loop<8>(rows, K, rot, u0, nu, all, first, stride, 256, isb, sink);
  else if (block == 512) mx_rotate_loop<16>(rows, K, rot, u0, nu, all, first, stride, 512, isb, sink);
  else mx_rotate_loop<32>(rows, K, rot, u0, nu, all, first, stride, 1024, isb, sink);
}

}  // namespace rq
