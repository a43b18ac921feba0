// MXFP4 products with many tokens: Y = A W^T on CTA pairs.
//
// The pair's 256 x 256 tile runs as tcgen05.mma.cta_group::2 kind::mxf4
// (M = 256): each CTA brings 128 token rows and 128 of the 256 weight rows per
// 256-wide K step, 35 KB for 512 cycles of MMA.  A single CTA's 128 x 256 tile
// needs 51 KB for as many, more than an SM takes from L2 in that time.
//
// Per CTA: warp 0 issues the copies, which count on the even CTA's barrier; warp
// 1 (even CTA) copies both CTAs' scales to TMEM and issues the pair's MMAs; warps
// 4-11 are the epilogue.  The accumulator takes 256 of the 512 TMEM columns and
// is single: the epilogue brings it into registers as packed BF16 first, hands
// it back, and stores while the next tile runs.
//
// 4608 x 12288 x 4096: 75-77 us, 6.0-6.2 PFLOP/s, tensor pipe 77% busy (87 under the
// power cap); a step of 256 columns takes 0.39 us, which is what its copies take
// without the MMAs (13 TB/s from L2 over all SMs; the MMAs 0.27).  65520 x 1536 x
// 8960: 370-400 us, 430-460 under the power cap, 0.8 of the 3.2 us a tile between
// its last MMA and the next tile's first.  Below about 1000 tokens most SMs are idle:
// K is not split, and 65 x 4096 x 4096 takes 16 pairs for 16 steps (10.4 us; the
// layer 12.4, that of 64 tokens, in rq_mxfew.cu, 10.6).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "rq_internal.h"
#include "rq_mx.cuh"
#include "rq_ptx.cuh"

namespace rq {

namespace {

constexpr int MG_THREADS = 384;
constexpr int MG_STAGES = 6;
constexpr int MG_SLOT_COLS = 24;         // TMEM columns of a stage's scales: 2 tiles of 4 for A, 4 for B
constexpr int MG_PA = 128 * 128, MG_PB = 128 * 128, MG_SA = 1024, MG_SB = 2048;
constexpr int MG_STAGE = MG_PA + MG_PB + MG_SA + MG_SB;
constexpr int MG_STG = 2048;             // an epilogue warp's 32 x 32 BF16 box
constexpr int MG_OFF_STG = MG_STAGES * MG_STAGE;
constexpr int MG_OFF_BAR = MG_OFF_STG + 8 * MG_STG;
constexpr int MG_BYTES = MG_OFF_BAR + 512;   // (no slack: the base has to be 1024-byte aligned)
static_assert(MG_BYTES <= 232448, "shared memory plan exceeds 227 KB");

struct __align__(64) MgMaps {
  CUtensorMap a, b;     // packed codes
  CUtensorMap sa, sb;   // scale tiles, 512 bytes a row
  CUtensorMap y;
};

struct MgParams {
  int M, N, K;
  void* Y;
  int out_fp32, tma_store;
  int32_t* status;
  uint64_t wait_ns;
  uint32_t inject_tx;
};

// M = 256 (bits 27-28), N = 256, E8M0 scales, scale bytes id and id + 1
__device__ __forceinline__ uint32_t mg_idesc(uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | (32u << 17) | (1u << 23) | (16u << 24) | (id << 29);
}

// 128 accumulator columns of this warp's 32 rows, from TMEM, as packed BF16; the
// loads go out two at a time (the MMAs wait for this)
__device__ __forceinline__ void mg_take(uint32_t acc, uint32_t (&w)[64]) {
#pragma unroll
  for (int ch = 0; ch < 4; ch += 2) {
    uint32_t v[2][32];
    tmem_ld32(acc + ch * 32, v[0]);
    tmem_ld32(acc + ch * 32 + 32, v[1]);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t* s = v[i / 16] + 2 * (i % 16);
      const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(s[0]), __uint_as_float(s[1]));
      w[ch * 16 + i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}
// ... to rows row0 .. row0 + 31, columns n0 .. n0 + 127 of Y by TMA stores of 32 x
// 32 boxes in shared memory
__device__ __forceinline__ void mg_store_tma(const MgParams& p, const CUtensorMap* ymap, const uint32_t (&w)[64],
                                             uint8_t* box, int row0, int n0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const int n = n0 + ch * 32;
    if (lane == 0) bulk_wait_group_read<0>();   // the last store has read the box
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c)   // 64-byte swizzle: 16-byte unit c of row r at unit c ^ (r / 2 % 4)
      *reinterpret_cast<uint4*>(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
          make_uint4(w[ch * 16 + 4 * c], w[ch * 16 + 4 * c + 1], w[ch * 16 + 4 * c + 2], w[ch * 16 + 4 * c + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      // rows >= M and columns >= N are clipped by the map; a box wholly outside is not stored
      if (row0 < p.M && n < p.N) tma_store_2d(ymap, smem_u32(box), n, row0);
      bulk_commit_group();
    }
  }
}
// ... when a row of Y is not a multiple of 16 bytes: through the box too, row by row
// with the lanes along it, two rows at a time for even N.  (Whole 16-byte units of
// Y, shifted into place, measured slower: 178 us against 149 at 6240 x 5120 x 9972,
// 145 against 149 at 15063 x 384 x 4511.)
__device__ __forceinline__ void mg_store_ragged(const MgParams& p, const uint32_t (&w)[64], uint8_t* box, int row0, int n0) {
  const int lane = threadIdx.x & 31, rows = min(32, p.M - row0);
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const int n = n0 + ch * 32;
    __syncwarp();   // (the box has been read)
#pragma unroll
    for (int c = 0; c < 4; ++c)   // 16-byte unit c of row r at unit c ^ (r / 2 % 4)
      *reinterpret_cast<uint4*>(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
          make_uint4(w[ch * 16 + 4 * c], w[ch * 16 + 4 * c + 1], w[ch * 16 + 4 * c + 2], w[ch * 16 + 4 * c + 3]);
    __syncwarp();
    uint16_t* out = static_cast<uint16_t*>(p.Y) + (size_t)row0 * p.N + n;
    if ((p.N & 1) == 0) {
      const int c = (lane & 15) * 2;   // (N even: n + c < N covers c + 1)
#pragma unroll 8
      for (int r = lane >> 4; r < rows; r += 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(box + r * 64 + (((c >> 3) ^ ((r >> 1) & 3)) << 4) + (c & 7) * 2);
        if (n + c < p.N) *reinterpret_cast<uint32_t*>(out + (size_t)r * p.N + c) = v;
      }
    } else {
#pragma unroll 8
      for (int r = 0; r < rows; ++r) {
        const uint16_t v = *reinterpret_cast<const uint16_t*>(box + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
        if (n + lane < p.N) out[(size_t)r * p.N + lane] = v;
      }
    }
  }
}
// FP32 output: 16 columns at a time through the box, half a warp along a row
__device__ __forceinline__ void mg_store_fp32(const MgParams& p, uint32_t acc, uint8_t* box, int row0, int n0) {
  const int lane = threadIdx.x & 31, c = lane & 15, rows = min(32, p.M - row0);
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    uint32_t v[32];
    tmem_ld32(acc + ch * 32, v);
    tmem_ld_wait();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + ch * 32 + h * 16;
      __syncwarp();   // (the box has been read)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4*>(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(v[h * 16 + 4 * q], v[h * 16 + 4 * q + 1], v[h * 16 + 4 * q + 2], v[h * 16 + 4 * q + 3]);
      __syncwarp();
      float* out = static_cast<float*>(p.Y) + (size_t)row0 * p.N + n;
#pragma unroll 4
      for (int r = lane >> 4; r < rows; r += 2) {
        const float y = *reinterpret_cast<const float*>(box + r * 64 + (((c >> 2) ^ ((r >> 1) & 3)) << 4) + (c & 3) * 4);
        if (n + c < p.N) out[(size_t)r * p.N + c] = y;
      }
    }
  }
}

__global__ void __launch_bounds__(MG_THREADS, 1) mx_gemm_kernel(const __grid_constant__ MgMaps tm,
                                                                const __grid_constant__ MgParams p) {
  extern __shared__ uint8_t smem[];
  if (smem_u32(smem) & 1023u) {   // (both CTAs see the same base)
    if (threadIdx.x == 0 && p.status) atomicCAS(p.status, 0, ST_SMEM_ALIGN);
    return;
  }
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + MG_OFF_BAR);   // even CTA: both CTAs' copies landed
  uint64_t* empty = full + MG_STAGES;      // the pair's MMAs have read the stage
  uint64_t* accfull = empty + MG_STAGES;
  uint64_t* accempty = accfull + 1;        // even CTA: both CTAs' epilogue warps have read the accumulator
  uint64_t* mdrain = accempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdrain + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const uint32_t rank = (uint32_t)uniform((int)cluster_ctarank());
  const int nk = (p.K + 255) / 256, KT = (p.K + 127) / 128;
  const int nN = (p.N + 255) / 256, ntiles = (p.M + 255) / 256 * nN;
  const int tile0 = (int)(blockIdx.x >> 1), tstep = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < MG_STAGES; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    mbar_init(accfull, 1);
    mbar_init(accempty, 16);
    mbar_init(mdrain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm.a);
    prefetch_tmap(&tm.b);
    prefetch_tmap(&tm.sa);
    prefetch_tmap(&tm.sb);
  }
  if (warp == 1) {
    tmem_alloc2(tmem_slot, 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers exist before either arrives on the other's
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  griddep_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    // both CTAs' copies count on the even CTA's barrier, which expects their sum
    uint32_t home;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(home) : "r"(smem_u32(full)));
    home = (uint32_t)uniform((int)home);
    const bool one = elect_one();
    int s = 0, ph = 0, filled = 0;   // stage, its phase, stages filled so far (up to all)
    bool ok = true, first = true;
    for (int tile = tile0; tile < ntiles && ok; tile += tstep) {
      const int m0 = tile / nN * 256 + (int)rank * 128, n0 = tile % nN * 256;
      const int sa0 = m0 / 128 * KT, sb0 = n0 / 128 * KT;
      for (int kt = 0; kt < nk; ++kt) {
        if (filled == MG_STAGES) {
          ok = warp_wait(&empty[s], ph ^ 1, p.status, ST_TIMEOUT_EMPTY, abort_flag, p.wait_ns);
          if (!ok) break;
        } else {
          ++filled;
        }
        if (one) {
          uint8_t* st = smem + s * MG_STAGE;
          if (rank == 0) mbar_expect_tx(&full[s], 2 * MG_STAGE + (first ? p.inject_tx : 0u));
          const uint32_t bar = home + s * 8;
          tma_load_2d_pair(st, &tm.a, kt * 128, m0, bar);
          tma_load_2d_pair(st + MG_PA, &tm.b, kt * 128, n0 + (int)rank * 128, bar);
          // two scale tiles per 128 rows (past the end: the next rows', or zeros, not used)
          tma_load_2d_pair(st + MG_PA + MG_PB, &tm.sa, 0, sa0 + kt * 2, bar);
#pragma unroll
          for (int b = 0; b < 2; ++b)   // each CTA multiplies all 256 weight rows
            tma_load_2d_pair(st + MG_PA + MG_PB + MG_SA + b * 1024, &tm.sb, 0, sb0 + b * KT + kt * 2, bar);
        }
        first = false;
        if (++s == MG_STAGES) { s = 0; ph ^= 1; }
      }
    }
    // this CTA's copies have landed once the MMAs have read them, and the last
    // commits arrive in this CTA's barriers: it may not leave before.  (s, ph):
    // the oldest of the stages still out, or with fewer than all filled, 0.
    if (filled < MG_STAGES) { s = 0; ph = 1; }
    for (int i = 0; i < filled; ++i) {
      if (ok)
        ok = warp_wait(&empty[s], ph ^ 1, p.status, ST_TIMEOUT_EMPTY, abort_flag, p.wait_ns);
      if (!ok && rank == 0)   // let the pair's copies land (bounded; the odd CTA waits at the end)
        mbar_drain(&full[s], ph ^ 1, p.wait_ns);
      if (++s == MG_STAGES) { s = 0; ph ^= 1; }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (rank == 0) {
      const bool one = elect_one();
      int s = 0, ph = 0, acc_ph = 1;
      // descriptors of the first stage; the address field counts 16-byte units
      const uint64_t d_op = smem_desc(sbase, 16, 1024, 2), d_sf = smem_desc(sbase + MG_PA + MG_PB, 16, 128, 0);
      // No branch is taken on a wait's answer: with one the compiler no longer takes
      // what follows for warp-uniform.  After a wait has run out the loop ends within
      // eight steps, but frees no stage any more: a copy into a stage whose last copies
      // are still out would arrive on a barrier that expects no arrival.
      bool ok = true;
      for (int tile = tile0; tile < ntiles; tile += tstep) {
        if (uniform(*abort_flag)) break;
        for (int kt = 0; kt < nk; ++kt) {
          ok &= mbar_wait_soon(&full[s], ph, p.status, ST_TIMEOUT_FULL, abort_flag, p.wait_ns);
          tc_fence_after();
          const uint32_t st = (uint32_t)(s * MG_STAGE) >> 4;
          // the scales to the stage's own TMEM columns, free again when the stage is
          const uint32_t tsf = tmem + 256 + s * MG_SLOT_COLS;
          if (one) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {   // 128 columns each; B: 8 TMEM columns of 256 rows
              tc_cp2_32x128b_warpx4(tsf + q * 4, d_sf + st + ((q * 512) >> 4));
#pragma unroll
              for (int b = 0; b < 2; ++b)
                tc_cp2_32x128b_warpx4(tsf + 8 + q * 8 + b * 4, d_sf + st + ((MG_SA + b * 1024 + q * 512) >> 4));
            }
          }
          if (kt == 0) {   // (the first tile finds the accumulator empty)
            ok &= mbar_wait_soon(accempty, acc_ph, p.status, ST_TIMEOUT_EPI, abort_flag, p.wait_ns);
            acc_ph ^= 1;
            tc_fence_after();
          }
          const int kkn = min(4, p.K / 64 - kt * 4);
          if (one) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (kk < kkn)
                umma_mxf4_2(tmem, d_op + st + ((kk * 32) >> 4), d_op + st + ((MG_PA + kk * 32) >> 4), mg_idesc((kk & 1) * 2),
                            tsf + (kk >> 1) * 4, tsf + 8 + (kk >> 1) * 8, kt > 0 || kk > 0);
            tc_commit2_mc_if(&empty[s], 0x3, ok);
            if (kt == nk - 1) tc_commit2_mc_if(accfull, 0x3, ok);
          }
          if (++s == MG_STAGES) { s = 0; ph ^= 1; }
          if ((kt & 7) == 7 && uniform(*abort_flag)) break;
        }
      }
      if (*abort_flag) {   // wait (bounded) for the MMAs issued
        if (one) tc_commit2_mc(mdrain, 0x1);
        mbar_drain(mdrain, 0, p.wait_ns);
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + half * 128;
    uint8_t* stg = smem + MG_OFF_STG + (warp - 4) * MG_STG;
    int tc = 0;
    bool ok = true;
    for (int tile = tile0; tile < ntiles && ok; tile += tstep, ++tc) {
      const int row0 = tile / nN * 256 + (int)rank * 128 + q * 32, n0 = tile % nN * 256 + half * 128;
      ok = warp_wait(accfull, tc & 1, p.status, ST_TIMEOUT_MMA, abort_flag, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      uint32_t w[64];
      if (p.out_fp32) mg_store_fp32(p, acc, stg, row0, n0);
      else mg_take(acc, w);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(accempty, 0);
      if (p.tma_store) mg_store_tma(p, &tm.y, w, stg, row0, n0);
      else if (!p.out_fp32) mg_store_ragged(p, w, stg, row0, n0);
    }
    if (lane == 0) bulk_wait_group<0>();   // the staging boxes outlive their stores
  }

  tc_fence_before();
  cluster_sync();   // neither CTA leaves while the other may still touch its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_mx_gemm(const GemmLaunch& a, cudaStream_t st, const char** why) {
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(mx_gemm_kernel));
  if (e != cudaSuccess) return e;
  MgMaps tm;
  MgParams p{};
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.Y = a.Y; p.out_fp32 = a.out_fp32;
  p.tma_store = !a.out_fp32 && a.N % 8 == 0;   // (the map's row pitch must be a multiple of 16 bytes)
  p.status = a.status; p.wait_ns = a.wait_ns; p.inject_tx = a.inject_tx;
  bool ok = mx_code_map(&tm.a, a.a_codes, a.M, a.K, 128) && mx_code_map(&tm.b, a.w_codes, a.N, a.K, 128) &&
            mx_scale_map(&tm.sa, a.a_bscale, a.M, a.K) && mx_scale_map(&tm.sb, a.w_bscale, a.N, a.K);
  if (p.tma_store) ok = ok && mx_out_map(&tm.y, a.Y, a.M, a.N);
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(MG_THREADS);
  cfg.dynamicSmemBytes = MG_BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;   // the occupancy query sees the cluster shape only
  // the pairs that can be resident at once, per device
  static std::atomic<int> resident[64];
  int dev = 0, pairs = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64) pairs = resident[dev].load();
  if (pairs < 1) {
    e = cudaOccupancyMaxActiveClusters(&pairs, mx_gemm_kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) resident[dev].store(pairs);
  }
  const int64_t tiles = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
  cfg.gridDim = dim3(2 * (unsigned)(tiles < pairs ? tiles : pairs));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, mx_gemm_kernel, tm, p);
}

}  // namespace rq
