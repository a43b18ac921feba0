// MXFP4 codes read back as the values they stand for.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rq_internal.h"
#include "rq_mx.cuh"

namespace rq {

namespace {

// One thread per 8 codes: a 4-byte read, a scale byte, 8 values out.
template <typename T>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* codes, const uint8_t* bscale, T* out,
                                                            int rows, int K) {
  const int words = K / 8;
  const int64_t n = (int64_t)rows * words;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int m = (int)(i / words), w = (int)(i % words);
    const uint32_t c = reinterpret_cast<const uint32_t*>(codes)[i];
    const float s = mx_scale(bscale[mx_sf_offset(m, w / 4, K)]);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[i * 8 + e] = (T)(e2m1_value((c >> (4 * e)) & 15u) * s);
  }
}

}  // namespace

cudaError_t launch_mx_dequantize(const MxDequantLaunch& a, cudaStream_t st) {
  const int64_t n = (int64_t)a.rows * (a.K / 8);
  const int64_t blocks = (n + 255) / 256, most = (int64_t)(a.num_sms > 0 ? a.num_sms : 148) * 16;
  const int grid = (int)(blocks < most ? blocks : most);
  if (a.out_fp32)
    mx_dequantize_kernel<float><<<grid, 256, 0, st>>>(a.codes, a.bscale, static_cast<float*>(a.out), a.rows, a.K);
  else
    mx_dequantize_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a.codes, a.bscale, static_cast<__nv_bfloat16*>(a.out), a.rows, a.K);
  return cudaGetLastError();
}

}  // namespace rq
