// MXFP4 products with many tokens: Y = A W^T on CTA pairs.
//
// The pair's 256 x 256 tile runs as tcgen05.mma.cta_group::2 kind::mxf4
// (M = 256): each CTA brings 128 token rows and 128 of the 256 weight rows per
// 256-wide K step, 35 KB for 512 cycles of MMA.  A single CTA's 128 x 256 tile
// needs 51 KB for as many, more than an SM takes from L2 in that time.
//
// Per CTA: warp 0 issues the copies; warp 1 the pair's MMAs (even CTA) or passes
// the odd CTA's landed stages on; warp 2 moves the scales to TMEM on an issue
// stream of its own (even CTA, both CTAs' tiles at once), a ring of slots ahead of
// the MMAs; warps 4-11 are the epilogue.  The accumulator takes 256 of the
// 512 TMEM columns and is single: the epilogue brings it into registers as
// packed BF16 first, hands it back, and stores while the next tile runs.
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
constexpr int MG_STAGES = 5;
constexpr int MG_SLOTS = 4;              // scale slots in TMEM
constexpr int MG_SLOT_COLS = 24;         // 2 scale tiles of 4 columns for A, 4 for B
constexpr int MG_PA = 128 * 128, MG_PB = 128 * 128, MG_SA = 1024, MG_SB = 2048;
constexpr int MG_STAGE = MG_PA + MG_PB + MG_SA + MG_SB;
constexpr int MG_STG = 4096;             // an epilogue warp's two 32 x 32 BF16 boxes
constexpr int MG_OFF_STG = MG_STAGES * MG_STAGE;
constexpr int MG_OFF_BAR = MG_OFF_STG + 8 * MG_STG;
constexpr int MG_BYTES = MG_OFF_BAR + 512 + 1024;
static_assert(MG_BYTES <= 232448, "shared memory plan exceeds 227 KB");

struct __align__(64) MgMaps {
  CUtensorMap a, b, y;
};

struct MgParams {
  int M, N, K;
  const uint8_t *a_sf, *w_sf;
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

__global__ void __launch_bounds__(MG_THREADS, 1) mx_gemm_kernel(const __grid_constant__ MgMaps tm,
                                                                const __grid_constant__ MgParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + MG_OFF_BAR);   // this CTA's copies landed
  uint64_t* pfull = full + MG_STAGES;      // even CTA: the odd CTA's copies landed
  uint64_t* empty = pfull + MG_STAGES;     // the pair's MMAs have read the stage
  uint64_t* sffull = empty + MG_STAGES;    // even CTA: scales in TMEM
  uint64_t* sfempty = sffull + MG_SLOTS;   // even CTA: MMAs done with a slot
  uint64_t* accfull = sfempty + MG_SLOTS;
  uint64_t* accempty = accfull + 1;        // even CTA: both CTAs' epilogue warps have read the accumulator
  uint64_t* mdrain = accempty + 1;
  uint64_t* cdrain = mdrain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cdrain + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int nk = (p.K + 255) / 256, KT = (p.K + 127) / 128;
  const int nN = (p.N + 255) / 256, ntiles = (p.M + 255) / 256 * nN;
  const int tile0 = (int)(blockIdx.x >> 1), tstep = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < MG_STAGES; ++i) { mbar_init(&full[i], 1); mbar_init(&pfull[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < MG_SLOTS; ++i) { mbar_init(&sffull[i], 1); mbar_init(&sfempty[i], 1); }
    mbar_init(accfull, 1);
    mbar_init(accempty, 16);
    mbar_init(mdrain, 1);
    mbar_init(cdrain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm.a);
    prefetch_tmap(&tm.b);
  }
  if (warp == 1) {
    tmem_alloc2(tmem_slot, 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers exist before either arrives on the other's
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t kc = 0;
      bool ok = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tstep) {
        const int m0 = tile / nN * 256 + (int)rank * 128, n0 = tile % nN * 256;
        // scale tiles exist for row tiles that hold a row
        const bool has_a = m0 < p.M;
        const int nb = min(2, (p.N + 127) / 128 - n0 / 128);
        for (int kt = 0; kt < nk; ++kt, ++kc) {
          const int s = kc % MG_STAGES;
          ok = (kc < (uint32_t)MG_STAGES ||
                mbar_wait(&empty[s], (kc / MG_STAGES - 1) & 1, p.status, ST_TIMEOUT_EMPTY, abort_flag, p.wait_ns)) &&
               !*abort_flag;
          if (!ok) break;
          uint8_t* st = smem + s * MG_STAGE;
          const uint32_t sfb = (uint32_t)min(2, KT - kt * 2) * 512;   // scale bytes of 128 rows
          mbar_expect_tx(&full[s], MG_PA + MG_PB + (nb + (has_a ? 1 : 0)) * sfb + (kc == 0 ? p.inject_tx : 0u));
          tma_load_2d(st, &tm.a, kt * 128, m0, &full[s]);
          tma_load_2d(st + MG_PA, &tm.b, kt * 128, n0 + (int)rank * 128, &full[s]);
          if (has_a) bulk_g2s(st + MG_PA + MG_PB, p.a_sf + ((size_t)(m0 / 128) * KT + kt * 2) * 512, sfb, &full[s]);
          for (int b = 0; b < nb; ++b)   // every CTA of the pair multiplies all 256 weight rows
            bulk_g2s(st + MG_PA + MG_PB + MG_SA + b * 1024, p.w_sf + ((size_t)(n0 / 128 + b) * KT + kt * 2) * 512, sfb, &full[s]);
        }
      }
      if (ok)   // the last commits land in this CTA's barriers: it may not leave before
        for (uint32_t c = kc > (uint32_t)MG_STAGES ? kc - MG_STAGES : 0; c < kc && ok; ++c)
          ok = mbar_wait(&empty[c % MG_STAGES], (c / MG_STAGES) & 1, p.status, ST_TIMEOUT_EMPTY, abort_flag, p.wait_ns);
      if (!ok)   // let the copies already issued land (bounded)
        for (uint32_t c = kc > (uint32_t)MG_STAGES ? kc - MG_STAGES : 0; c < kc; ++c)
          mbar_drain(&full[c % MG_STAGES], (c / MG_STAGES) & 1, p.wait_ns);
    }
  } else if (warp == 1 && rank == 1) {
    // ------------------------------------------------------------ the odd CTA's stages, passed on
    if (lane == 0) {
      uint32_t kc = 0;
      bool ok = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tstep)
        for (int kt = 0; kt < nk && ok; ++kt, ++kc) {
          const int s = kc % MG_STAGES;
          ok = mbar_wait(&full[s], (kc / MG_STAGES) & 1, p.status, ST_TIMEOUT_FULL, abort_flag, p.wait_ns);
          if (ok) mbar_arrive_cluster(&pfull[s], 0);
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t kc = 0;
      int tc = 0;
      bool ok = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tstep, ++tc) {
        ok = tc == 0 || mbar_wait(accempty, (tc - 1) & 1, p.status, ST_TIMEOUT_EPI, abort_flag, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        for (int kt = 0; kt < nk; ++kt, ++kc) {
          const int s = kc % MG_STAGES, sl = kc % MG_SLOTS;
          ok = mbar_wait(&full[s], (kc / MG_STAGES) & 1, p.status, ST_TIMEOUT_FULL, abort_flag, p.wait_ns) &&
               mbar_wait(&pfull[s], (kc / MG_STAGES) & 1, p.status, ST_TIMEOUT_FULL, abort_flag, p.wait_ns) &&
               mbar_wait(&sffull[sl], (kc / MG_SLOTS) & 1, p.status, ST_TIMEOUT_FULL, abort_flag, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint32_t st = sbase + s * MG_STAGE, tsf = tmem + 256 + sl * MG_SLOT_COLS;
          const int kkn = min(4, p.K / 64 - kt * 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (kk < kkn)
              umma_mxf4_2(tmem, smem_desc(st + kk * 32, 16, 1024, 2), smem_desc(st + MG_PA + kk * 32, 16, 1024, 2),
                          mg_idesc((kk & 1) * 2), tsf + (kk >> 1) * 4, tsf + 8 + (kk >> 1) * 8, kt > 0 || kk > 0);
          tc_commit2_mc(&empty[s], 0x3);
          tc_commit2_mc(&sfempty[sl], 0x1);
        }
        if (ok) tc_commit2_mc(accfull, 0x3);
      }
      if (!ok) {   // wait (bounded) for the MMAs already issued
        tc_commit2_mc(mdrain, 0x1);
        mbar_drain(mdrain, 0, p.wait_ns);
      }
    }
  } else if (warp == 2 && rank == 0) {
    // ------------------------------------------------------------ scales -> TMEM, in both CTAs
    if (lane == 0) {
      uint32_t kc = 0;
      bool ok = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tstep)
        for (int kt = 0; kt < nk; ++kt, ++kc) {
          const int s = kc % MG_STAGES, sl = kc % MG_SLOTS;
          ok = (kc < (uint32_t)MG_SLOTS ||
                mbar_wait(&sfempty[sl], (kc / MG_SLOTS - 1) & 1, p.status, ST_TIMEOUT_EMPTY, abort_flag, p.wait_ns)) &&
               mbar_wait(&full[s], (kc / MG_STAGES) & 1, p.status, ST_TIMEOUT_FULL, abort_flag, p.wait_ns) &&
               mbar_wait(&pfull[s], (kc / MG_STAGES) & 1, p.status, ST_TIMEOUT_FULL, abort_flag, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sf = sbase + s * MG_STAGE + MG_PA + MG_PB, tsf = tmem + 256 + sl * MG_SLOT_COLS;
#pragma unroll
          for (int q = 0; q < 2; ++q) {   // 128 columns each; B: 8 TMEM columns of 256 rows
            tc_cp2_32x128b_warpx4(tsf + q * 4, smem_desc(sf + q * 512, 16, 128, 0));
#pragma unroll
            for (int b = 0; b < 2; ++b)
              tc_cp2_32x128b_warpx4(tsf + 8 + q * 8 + b * 4, smem_desc(sf + MG_SA + b * 1024 + q * 512, 16, 128, 0));
          }
          tc_commit2_mc(&sffull[sl], 0x1);
        }
      if (!ok) {
        tc_commit2_mc(cdrain, 0x1);
        mbar_drain(cdrain, 0, p.wait_ns);
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + half * 128;
    const uint32_t stg = sbase + MG_OFF_STG + (warp - 4) * MG_STG;
    int tc = 0;
    bool ok = true;
    for (int tile = tile0; tile < ntiles && ok; tile += tstep, ++tc) {
      const int row0 = tile / nN * 256 + (int)rank * 128 + q * 32, n0 = tile % nN * 256 + half * 128;
      ok = mbar_wait(accfull, tc & 1, p.status, ST_TIMEOUT_MMA, abort_flag, p.wait_ns);
      if (!ok) break;
      tc_fence_after();
      if (p.out_fp32) {
        const int row = row0 + lane;
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t v[32];
          tmem_ld32(acc + ch * 32, v);
          tmem_ld_wait();
          float* out = static_cast<float*>(p.Y) + (size_t)row * p.N + n0 + ch * 32;
          if (row < p.M) {
            if (n0 + ch * 32 + 32 <= p.N && (p.N & 3) == 0) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<uint4*>(out + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (n0 + ch * 32 + i < p.N) out[i] = __uint_as_float(v[i]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(accempty, 0);
        continue;
      }
      // BF16: the warp's 32 x 128 values into registers, two to a word, and the
      // accumulator back to the MMAs
      uint32_t w[64];
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t v[32];
        tmem_ld32(acc + ch * 32, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
          w[ch * 16 + i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(accempty, 0);
      if (p.tma_store) {
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          // two boxes in turn: the store two back has read this one
          const uint32_t buf = stg + (ch & 1) * 2048;
          if (lane == 0) bulk_wait_group_read<1>();
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 4; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)),
                         "r"(w[ch * 16 + 4 * c]), "r"(w[ch * 16 + 4 * c + 1]), "r"(w[ch * 16 + 4 * c + 2]),
                         "r"(w[ch * 16 + 4 * c + 3])
                         : "memory");
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            // rows >= M and columns >= N are clipped by the map; a box wholly outside is not stored
            if (row0 < p.M && n0 + ch * 32 < p.N) tma_store_2d(&tm.y, buf, n0 + ch * 32, row0);
            bulk_commit_group();
          }
        }
      } else if (row0 + lane < p.M) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.Y) + (size_t)(row0 + lane) * p.N + n0;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
          if (n0 + 2 * i < p.N) out[2 * i] = h.x;
          if (n0 + 2 * i + 1 < p.N) out[2 * i + 1] = h.y;
        }
      }
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
  p.a_sf = a.a_bscale; p.w_sf = a.w_bscale;
  p.Y = a.Y; p.out_fp32 = a.out_fp32;
  p.tma_store = !a.out_fp32 && a.N % 8 == 0;   // (the map's row pitch must be a multiple of 16 bytes)
  p.status = a.status; p.wait_ns = a.wait_ns; p.inject_tx = a.inject_tx;
  bool ok = mx_code_map(&tm.a, a.a_codes, a.M, a.K, 128) && mx_code_map(&tm.b, a.w_codes, a.N, a.K, 128);
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
