// Internal launch descriptors shared by the C-ABI layer and the kernels.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#define RQ_FMT_INT4 1
#define RQ_FMT_LM16 2
#define RQ_FMT_NVFP4 3
#define RQ_FMT_LM4 4
#define RQ_FMT_INT4A 5
#define RQ_FMT_INT8 6
#define RQ_FMT_MXFP4 7

namespace rq {

struct K1Launch {
  int fmt;
  int weight;              // 1: weight rows (INT4 per-128-group scales, L = W U)
  const uint16_t* x;
  int rows, K, block;
  const int32_t* rot;
  const int32_t* rot2;     // double rotation: the second rotation's table, or null
  float inv_sqrt_b, sqrtK;
  int nbnd;
  const float* bnd;        // host, nbnd entries
  const uint16_t* U;
  int r;
  uint16_t* coef;
  uint8_t* codes;
  float* scale;
  float* zp;               // asymmetric INT4: per-row zero point
  float* wz;               // INT4 weights: per-row sum over groups of scale x code sum (or null)
  uint8_t* bscale;
  int32_t* status;
  int num_sms;
  uint64_t wait_ns;        // bounded-wait limit of every mbarrier wait
  uint32_t inject_tx;      // test hook: extra expect-tx bytes on the first load (0: off)
};

cudaError_t launch_k1(const K1Launch& a, cudaStream_t st);
// the rows-as-lanes activation kernel (every case without the projection)
bool k1r_supports(const K1Launch& a);
cudaError_t launch_k1r(const K1Launch& a, cudaStream_t st);

struct GemmLaunch {
  int a_fmt, w_fmt;
  int M, N, K;
  const uint8_t* a_codes;
  const float* a_scale;
  const uint8_t* a_bscale;
  const uint8_t* w_codes;
  const float* w_scale;
  const uint8_t* w_bscale;
  uint8_t a_lut[16];       // e4m3 bytes per code (FP8 path)
  uint8_t w_lut[16];
  const float* a_zp;       // asymmetric INT4 activations: per-token zero point (or null)
  const float* w_zsum;     // with a_zp: per weight row, sum_g s_w[g, n] * sum_{k in g} q_w[n, k]
  const uint16_t* c;       // M x r BF16 (low-rank branch) or null
  const uint16_t* L;       // N x r BF16
  int r;
  void* Y;
  int out_fp32;
  int early_weights;       // MXFP4, few tokens: the kernel before this one on the stream does not write the
                           // weights and started after everything before it had finished
  int32_t* status;
  int num_sms;
  uint64_t wait_ns;
  uint32_t inject_tx;
};

cudaError_t launch_gemm(const GemmLaunch& a, cudaStream_t st, const char** why);
// W8A8: 8-bit per-token activations x 8-bit per-channel weights (no expansion)
cudaError_t launch_gemm_w8a8(const GemmLaunch& a, cudaStream_t st);

// DiRotQ full PCA rotation: y = x V (FP32, into the caller's workspace), then
// the first r coordinates to BF16 and the rest to INT4.
struct PcaLaunch {
  int weight;              // 1: weight rows (one INT4 scale per 128 coordinates)
  const uint16_t* x;       // rows x K BF16
  const uint16_t* vt;      // K x K BF16, row n = column n of V
  int rows, K, r;
  float* y;                // rows x K FP32 workspace
  uint16_t* coef;          // rows x r BF16
  uint8_t* codes;          // rows x K/2
  float* scale;            // rows (activations) or K/128 x rows (weights)
  int32_t* status;
  int num_sms;
  uint64_t wait_ns;
};

cudaError_t launch_pca(const PcaLaunch& a, cudaStream_t st);

// Raises a kernel's dynamic shared memory limit to the most a CTA can have,
// once per device.
struct SmemLimit {
  std::atomic<uint64_t> done{0};
  cudaError_t raise(const void* kernel) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1u))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
  }
};

// MXFP4 rows with one rotation and no low-rank branch (rq_mx.cu)
cudaError_t launch_mx_quantize(const K1Launch& a, cudaStream_t st);
// MXFP4 codes -> values
struct MxDequantLaunch {
  const uint8_t* codes;
  const uint8_t* bscale;
  void* out;
  int rows, K, out_fp32, num_sms;
};
cudaError_t launch_mx_dequantize(const MxDequantLaunch& a, cudaStream_t st);

// mixture-of-experts layer on MXFP4 experts (at most 64 tokens)
struct MoeLaunch {
  int T, K, I, E, top_k, renorm, block, block2, out_fp32;
  const uint16_t* x;
  const uint16_t* router;
  const int32_t* rot;
  const uint8_t *w1, *w1_sf, *w2, *w2_sf;
  int32_t* idx;
  float* wts;
  uint8_t* ws;
  void* Y;
  float inv_sqrt_b, inv_sqrt_b2;
  int32_t* status;
  int num_sms;
  uint64_t wait_ns;
  uint32_t inject_tx;
};
// Tensor maps: packed codes, rows x cols / 2 bytes in boxes of 128 bytes x
// box_rows; scale tiles, 512 bytes a row, in pairs; BF16 output in 32 x 32 boxes (64-byte swizzle, cols % 8 == 0)
bool mx_code_map(CUtensorMap* m, const uint8_t* codes, uint64_t rows, uint64_t cols, uint32_t box_rows);
bool mx_scale_map(CUtensorMap* m, const uint8_t* sf, uint64_t rows, uint64_t cols);
bool mx_out_map(CUtensorMap* m, void* Y, uint64_t rows, uint64_t cols);
// MXFP4 products of more tokens, without the low-rank branch (rq_mxgemm.cu)
cudaError_t launch_mx_gemm(const GemmLaunch& a, cudaStream_t st, const char** why);
// MXFP4 products of at most MX_FEW_TOKENS tokens (rq_mxfew.cu); with the low-rank
// branch only where mx_few_low_rank says so
constexpr int MX_FEW_TOKENS = 64;
bool mx_few_low_rank(int M, int N, int K, int r, int sms);
cudaError_t launch_mx_few(const GemmLaunch& a, cudaStream_t st, const char** why);
// the whole layer from BF16 rows in one launch, for the shapes it takes
bool mx_layer_fused(int M, int N, int K, int sms);
cudaError_t launch_mx_layer_fused(const GemmLaunch& a, const uint16_t* x, const int32_t* rot, int block, float inv_sqrt_b,
                                  cudaStream_t st);
// gate/up and down products of an expert layer whose routing and activation
// codes are in place; `active`: the most experts that T tokens can choose
cudaError_t launch_moe_products(const MoeLaunch& a, const uint8_t* xq, const uint8_t* xq_sf, uint8_t* hq, uint8_t* hq_sf,
                                int active, cudaStream_t st);
size_t moe_workspace_bytes(int T, int K, int I, int E, int top_k);
cudaError_t launch_moe(const MoeLaunch& a, cudaStream_t st);

}  // namespace rq
