// MXFP4 pieces shared by the kernels: blocks of 32 values held as E2M1
// elements times a power of two, 2^(byte - 127) (E8M0; OCP Microscaling
// specification), scale bytes in 128-row x 128-column tiles of 512 bytes.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

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

}  // namespace rq
