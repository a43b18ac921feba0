// MXFP4 products with few tokens: the weights on the tensor core's M side.
//
// With T <= 64 tokens a product is bound by reading its weights once (17/32 of
// a byte each).  A tile of tokens x weights with the tokens on the M side would
// waste 128 - T of its rows and leave N / 256 CTAs to read everything; here 128
// weight rows are the M side of tcgen05.mma kind::mxf4 and the tokens its N
// (16, 32, 48 or 64), and the contraction is split over the CTAs of a cluster,
// which join their FP32 partial sums through distributed shared memory, always
// in rank order.
//
// One mainloop, four uses:
//   LINEAR   Y[t, n] = sum_k W[n, k] x[t, k] (+ c L^T)
//   FUSED    the same from BF16 rows: each CTA transforms and quantizes its own
//            part of the rows while the weights are on their way, which costs
//            less than a launch of its own (a few thousand values per CTA)
//   GATE_UP  one active expert and 128 hidden channels per cluster: two
//            accumulators (gate rows, up rows); h = w silu(g) u, the block
//            Hadamard transform and the MXFP4 quantization of the hidden rows in
//            the epilogue, where the 128 channels of a token are one warp's
//   DOWN     the contraction runs over all active experts one after another;
//            hidden rows of tokens that did not choose an expert are zeros, so
//            the sum over a token's experts happens in the accumulator
//
// Bound by the bytes of the weights where there are many (64 tokens, 128 experts of
// 2048 x 768, top 8: 82 us for the layer, of which 48 are the bytes; gate/up about
// 40, down 25), by latencies where there are few (1 x 4096 x 12288, fused: 10.9 us
// of which the weights' bytes are 4.1).
//
// Per CTA: warp 0 issues the copies (weights and tokens by TMA, 256 columns =
// 128 bytes a row per stage; scale tiles by bulk copies), warp 1 moves the
// scales to TMEM and issues the MMAs, warps 4-7 drain the accumulator, all
// warps do the epilogue.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "rq_internal.h"
#include "rq_mx.cuh"
#include "rq_ptx.cuh"

namespace rq {

namespace {

constexpr int FEW_THREADS = 256;
constexpr int FEW_MAX_STAGES = 8;
constexpr int FEW_PITCH = 132;          // floats between tokens of the partial sums (16-byte rows, no bank repeats)
constexpr int FEW_TAIL = 2048;          // barriers, TMEM address, active experts, the expert's tokens

struct __align__(64) FewMaps {
  CUtensorMap w;   // weight codes, all experts' rows one after another
  CUtensorMap x;   // token codes
};

struct FewParams {
  int T, NT;               // tokens; the MMA's N, T rounded up to 16
  int K;                   // contraction length (of one expert)
  int N;                   // output rows (LINEAR, DOWN) or hidden channels I (GATE_UP)
  int stages;
  int tail;                // offset of the barriers, behind the stages
  uint32_t tmem_cols;
  int early;               // weights may be read before the previous kernel has finished
  const uint8_t* w_sf;     // weight scales: of one expert after another
  size_t w_sf_expert;      // bytes of one expert's scales
  const uint8_t* x_sf;     // token scales (DOWN: one buffer per active expert)
  const int32_t* idx;      // T x top_k chosen experts
  const float* wts;
  int top_k;
  const uint16_t *c, *L;   // low-rank branch (LINEAR)
  int r;
  void* Y;
  int out_fp32;
  uint8_t *hq, *hq_sf;     // hidden rows out (GATE_UP)
  int block2;
  float inv_sqrt_b2;
  const uint16_t* xb;      // FUSED: T x K BF16 rows, their rotation, offsets in shared memory of the
  const int32_t* rot;      // codes of all steps (the scales behind them), rows and table entries
  int block, off_x, off_rows, off_rot;
  float inv_sqrt_b;
  int32_t* status;
  uint64_t wait_ns;
  uint32_t inject_tx;
};

__device__ __forceinline__ uint32_t few_mapa(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 few_ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void few_tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Ascending list of the experts that some token chose, in act[]; its length.
// flag: 256 bytes, words: 8 words of shared scratch.  Called by the whole CTA.
__device__ int list_active(const int32_t* idx, int n, uint8_t* flag, uint32_t* words, uint16_t* act) {
  const int e = (int)threadIdx.x;   // 256 threads, one expert each
  flag[e] = 0;
  __syncthreads();
  for (int i = e; i < n; i += FEW_THREADS) flag[__ldcg(idx + i) & 255] = 1;
  __syncthreads();
  const uint32_t w = __ballot_sync(0xffffffffu, flag[e]);
  if ((e & 31) == 0) words[e >> 5] = w;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = __popc(words[i]);
    before += i < (e >> 5) ? c : 0;
    all += c;
  }
  if (flag[e]) act[before + __popc(w & ((1u << (e & 31)) - 1u))] = (uint16_t)e;
  __syncthreads();
  return all;
}

// E2M1 x E2M1, E8M0 scales per 32, N = n; a 64-wide instruction takes bytes
// id, id + 1 of each scale word.
__device__ __forceinline__ uint32_t few_idesc(int n, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | (8u << 24) | (id << 29);
}

enum { LINEAR = 0, GATE_UP = 1, DOWN = 2, FUSED = 3 };
constexpr int FUSED_SF = 512;           // FUSED: scale bytes per step, two tiles 256 bytes apart: the rows past
                                        // the 16th that a tile's copy also brings are other tiles', not used
constexpr int FUSED_MIN_STAGES = 3;     // see launch_mode
constexpr int FUSED_THREADS = 384;
constexpr int FUSED_WARPS = FUSED_THREADS / 32 - 2;   // all but the first two transform the rows
__host__ __device__ constexpr int few_threads(int mode) { return mode == FUSED ? FUSED_THREADS : FEW_THREADS; }

template <int MODE>
__global__ void __launch_bounds__(few_threads(MODE), 2) mx_few_kernel(const __grid_constant__ FewMaps tm,
                                                                const __grid_constant__ FewParams p) {
  constexpr int NA = MODE == GATE_UP ? 2 : 1;
  constexpr int PA = 128 * 128, SF = 1024;            // weight codes, scales of 128 rows per stage
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const int PB = p.NT * 128;
  constexpr bool EXPERTS = MODE == GATE_UP || MODE == DOWN;
  const int STAGE = NA * (PA + SF) + (MODE == FUSED ? 0 : PB + SF);
  // stage: [NA] weight codes | token codes | [NA] weight scales | token scales
  uint8_t* tail = smem + p.tail;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* empty = full + FEW_MAX_STAGES;
  uint64_t* accfull = empty + FEW_MAX_STAGES;
  uint64_t* mdrain = accfull + 1;
  uint64_t* xready = mdrain + 1;          // FUSED: the rows are quantized
  uint64_t* xfull = xready + 1;           // FUSED: the rows and the table are here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(xfull + 1);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  uint32_t* words = tmem_slot + 4;
  uint16_t* act = reinterpret_cast<uint16_t*>(words + 8);
  uint8_t* flag = reinterpret_cast<uint8_t*>(act + 256);   // GATE_UP reuses it: the tokens that chose the expert
  float* wsel = reinterpret_cast<float*>(flag + 256);      // and their weights
  float* part = reinterpret_cast<float*>(smem);       // [NA][NT][FEW_PITCH], over the stages once they are used up

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  uint32_t S;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  S = (uint32_t)uniform((int)S);
  const uint32_t rank = (uint32_t)uniform((int)cluster_ctarank());
  const int tile = (int)(blockIdx.x / S), n0 = tile * 128;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    mbar_init(accfull, 1);
    mbar_init(mdrain, 1);
    mbar_init(xready, FUSED_WARPS);
    mbar_init(xfull, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm.w);
    if (MODE != FUSED) prefetch_tmap(&tm.x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  if (!p.early) griddep_wait();

  // this rank's steps of 256 columns: [s0, s0 + n)
  const int spe = (p.K + 255) / 256, KT = (p.K + 127) / 128;
  int total = spe, expert = 0;
  bool live = true;
  if constexpr (EXPERTS) {
    const int na = uniform(list_active(p.idx, p.T * p.top_k, flag, words, act));
    if constexpr (MODE == GATE_UP) {
      griddep_launch_dependents();   // every CTA of this grid has seen the routing by now
      live = (int)blockIdx.y < na;
      if (live) expert = uniform(act[blockIdx.y]);
    } else {
      total = na * spe;
    }
  }
  const int s0 = (int)((int64_t)total * rank / S);
  const int n = live ? (int)((int64_t)total * (rank + 1) / S) - s0 : 0;

  if (warp == 0) {
    const bool one = elect_one();
    const size_t rowt = (size_t)(n0 / 128) * KT * 512;   // this row tile's scales
    // position of a step: stage and its phase, K step of the expert, place in
    // the list of active experts (counted on: a division costs more than the rest)
    struct Pos { int s, ph, kt, a; };
    auto next = [&](Pos& q) {
      if (++q.s == p.stages) { q.s = 0; q.ph ^= 1; }
      if (++q.kt == spe) { q.kt = 0; ++q.a; }
    };
    auto load = [&](const Pos& q, bool first, bool wt, bool tk) {
      const int e = MODE == DOWN ? uniform(act[q.a]) : expert;
      if (!one) return;
      uint64_t* bar = &full[q.s];
      uint8_t* s = smem + q.s * STAGE;
      const uint32_t sfb = (uint32_t)min(2, KT - q.kt * 2) * 512;   // scale bytes of 128 rows
      if (wt) {
        mbar_expect_tx(bar, NA * (PA + sfb) + (MODE == FUSED ? 0 : PB + sfb) + (first ? p.inject_tx : 0u));
        const uint8_t* sf = p.w_sf + (EXPERTS ? (size_t)e * p.w_sf_expert : 0) + (size_t)q.kt * 1024;
#pragma unroll
        for (int h = 0; h < NA; ++h) {   // GATE_UP: rows I..2I-1 are the up rows
          const int row = (EXPERTS ? e * NA * p.N : 0) + h * p.N + n0;
          tma_load_2d(s + h * PA, &tm.w, q.kt * 128, row, bar);
          bulk_g2s(s + NA * PA + (MODE == FUSED ? 0 : PB) + h * SF, sf + (size_t)h * (p.N / 128) * KT * 512 + rowt, sfb, bar);
        }
      }
      if (MODE != FUSED && tk) {
        const int a = MODE == DOWN ? q.a : 0;
        tma_load_2d(s + NA * PA, &tm.x, q.kt * 128, a * p.T, bar);
        bulk_g2s(s + NA * (PA + SF) + PB, p.x_sf + (size_t)a * KT * 512 + (size_t)q.kt * 1024, sfb, bar);
      }
    };
    if (MODE == FUSED && one) {   // the rows, and the table's entries of this rank's columns (whole Hadamard blocks)
      const int U = p.block < 64 ? 64 : p.block;
      const int u0 = s0 * 256 / U, u1 = (min(p.K, (s0 + n) * 256) + U - 1) / U;
      if (n > 0) {
        mbar_expect_tx(xfull, (uint32_t)(p.T * p.K * 2 + (u1 - u0) * U * 4));
        bulk_g2s(smem + p.off_rot, p.rot + u0 * U, (uint32_t)(u1 - u0) * U * 4, xfull);
        bulk_g2s(smem + p.off_rows, p.xb, (uint32_t)(p.T * p.K * 2), xfull);
      }
    }
    Pos q{0, 0, s0 % spe, s0 / spe};
    int i = 0;
    if (p.early) {   // the first stages' weights now, their tokens once the previous kernel is done
      const int head = min(n, p.stages);
      const Pos q0 = q;
      for (int j = 0; j < head; ++j) { load(q, j == 0, true, false); next(q); }
      griddep_wait();
      q = q0;
      for (; i < head; ++i) { load(q, false, false, true); next(q); }
    }
    for (; i < n; ++i) {
      if (i >= p.stages && !warp_wait(&empty[q.s], q.ph ^ 1, p.status, ST_TIMEOUT_EMPTY, abort_flag, p.wait_ns)) break;
      load(q, i == 0, true, true);
      next(q);
    }
    if (MODE == FUSED && n > 0 && *abort_flag) mbar_drain(xfull, 0, p.wait_ns);
    if (i < n)   // let the copies already issued land (bounded)
      for (int j = i > p.stages ? i - p.stages : 0; j < i; ++j) mbar_drain(&full[j % p.stages], (j / p.stages) & 1, p.wait_ns);
  } else if (warp == 1) {
    if (n > 0) {
      const bool one = elect_one();
      int s = 0, ph = 0, kt = s0 % spe;
      // descriptors of the first stage; the address field counts 16-byte units,
      // so everything else is one addition (rebuilding them for every
      // instruction took 150 of 550 cycles a step)
      const uint64_t d_op = smem_desc(sbase, 16, 1024, 2), d_sf = smem_desc(sbase + NA * PA + (MODE == FUSED ? 0 : PB), 16, 128, 0);
      const uint64_t d_x = smem_desc(sbase + (MODE == FUSED ? p.off_x : NA * PA), 16, 1024, 2);
      const uint64_t d_xsf = smem_desc(sbase + (MODE == FUSED ? p.off_x + n * PB : NA * PA + PB + NA * SF), 16, 128, 0);
      // No branch is taken on a wait's answer: with one the compiler no longer takes
      // what follows for warp-uniform.  After a wait has run out the loop ends within
      // eight steps on whatever is there, but frees no stage any more: a copy into a stage
      // whose last copies are still out would arrive on a barrier that expects no arrival.
      bool ok = true;
      if (MODE == FUSED) ok = mbar_wait_soon(xready, 0, p.status, ST_TIMEOUT_FULL, abort_flag, p.wait_ns);
      const uint32_t id0 = few_idesc(p.NT, 0), id2 = few_idesc(p.NT, 2);
      for (int i = 0; i < n; ++i) {
        ok &= mbar_wait_soon(&full[s], ph, p.status, ST_TIMEOUT_FULL, abort_flag, p.wait_ns);
        tc_fence_after();
        const int sct = min(2, KT - kt * 2), kkn = min(4, p.K / 64 - kt * 4);
        const uint32_t st = (uint32_t)(s * STAGE) >> 4;
        const uint32_t xst = MODE == FUSED ? (uint32_t)(i * PB) >> 4 : st;          // token codes and scales:
        const uint32_t xsf = MODE == FUSED ? (uint32_t)(i * FUSED_SF) >> 4 : st;    // of every step, or the stage's
        // a slot of scale columns per stage: free again when the stage is
        const uint32_t tsf = tmem + NA * p.NT + s * (NA + 1) * 8;
        if (one) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            if (q < sct) {
#pragma unroll
              for (int h = 0; h < NA; ++h) tc_cp_32x128b_warpx4(tsf + h * 8 + q * 4, d_sf + st + ((h * SF + q * 512) >> 4));
              tc_cp_32x128b_warpx4(tsf + NA * 8 + q * 4, d_xsf + xsf + ((q * (MODE == FUSED ? 256 : 512)) >> 4));
            }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (kk < kkn) {
#pragma unroll
              for (int h = 0; h < NA; ++h)
                umma_mxf4(tmem + h * p.NT, d_op + st + ((h * PA + kk * 32) >> 4), d_x + xst + ((kk * 32) >> 4),
                          kk & 1 ? id2 : id0, tsf + h * 8 + (kk >> 1) * 4, tsf + NA * 8 + (kk >> 1) * 4, i > 0 || kk > 0);
            }
          tc_commit_if(&empty[s], ok);
          if (i == n - 1) tc_commit_if(accfull, ok);
        }
        if (++s == p.stages) { s = 0; ph ^= 1; }
        if (++kt == spe) kt = 0;
        // (FUSED has at most 32 steps; there the look costs 0.1 of 10.9 us)
        if (MODE != FUSED && (i & 7) == 7 && uniform(*abort_flag)) break;
      }
      if (*abort_flag) {   // wait (bounded) for the MMAs issued
        if (one) tc_commit(mdrain);
        mbar_drain(mdrain, 0, p.wait_ns);
      }
    }
  } else if (MODE == GATE_UP && warp < 4) {
    // ------------------------------------------------------------ the expert's tokens
    // while the weights stream: whether each token chose the expert and its
    // weight, and zeros (codes and scale bytes) into this tile's hidden rows of
    // the others; each rank of the cluster the tokens t % S
    const int t = (warp - 2) * 32 + lane;
    if (t < 64) {
      uint8_t hit = 0;
      if (live && t < p.T)
        for (int j = 0; j < p.top_k; ++j)
          if (__ldcg(p.idx + t * p.top_k + j) == expert) {
            hit = 1;
            wsel[t] = __ldcg(p.wts + t * p.top_k + j);
          }
      flag[t] = hit;
      if (live && t < p.T && !hit && t % (int)S == (int)rank) {
        uint4* row = reinterpret_cast<uint4*>(p.hq + ((size_t)blockIdx.y * p.T + t) * (p.N / 2) + n0 / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint32_t*>(p.hq_sf + (size_t)blockIdx.y * (p.N / 128) * 512 + mx_sf_offset(t, n0 / 32, p.N)) = 0u;
      }
    }
  }
  if constexpr (MODE == FUSED) {
    if (warp >= 2) {
      // ------------------------------------------------------------ rotate + quantize
      // this rank's columns [c0, c1) of every row, from whole Hadamard blocks
      const int c0 = s0 * 256, c1 = min(p.K, (s0 + n) * 256), U = p.block < 64 ? 64 : p.block;
      const int u0 = c0 / U, u1 = (c1 + U - 1) / U;
      const uint16_t* rows = reinterpret_cast<const uint16_t*>(smem + p.off_rows);
      const int32_t* rot = reinterpret_cast<const int32_t*>(smem + p.off_rot);
      const bool ok = n > 0 && warp_wait(xfull, 0, p.status, ST_TIMEOUT_LOAD, abort_flag, p.wait_ns);
      const int nu = ok ? u1 - u0 : 0;
      const auto sink = [&](int t, int k, uint8_t*& codes, uint8_t*& sf) {
        if (k < c0 || k >= c1) return false;
        const int c = k - c0, step = c >> 8, byte = (c & 255) >> 1;
        // 128-byte swizzle: 16-byte unit j of row t at unit j ^ (t % 8)
        codes = smem + p.off_x + step * PB + t * 128 + (((byte >> 4) ^ (t & 7)) << 4) + (byte & 15);
        sf = smem + p.off_x + n * PB + step * FUSED_SF + ((c & 255) >> 7) * 256 + t * 16 + ((c >> 5) & 3);
        return true;
      };
      mx_rotate_units(rows, p.K, rot, u0, nu, nu * p.T, warp - 2, FUSED_WARPS, p.block, p.inv_sqrt_b, sink);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(xready);
    }
  }
  if (warp >= 4 && warp < 8) {
    const int q = warp & 3;
    const bool ok = n > 0 && warp_wait(accfull, 0, p.status, ST_TIMEOUT_MMA, abort_flag, p.wait_ns);
    if (ok) tc_fence_after();
    for (int c = 0; c < NA * p.NT; c += 16) {
      uint32_t v[16];
      if (ok) {
        few_tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c, v);
        tmem_ld_wait();
      } else {   // no steps fell to this rank
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0u;
      }
      if (ok || n == 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * FEW_PITCH + q * 32 + lane] = __uint_as_float(v[j]);
      }
    }
    tc_fence_before();
  }
  if (p.early) griddep_wait();   // nothing is written before the previous kernel is done
  __syncwarp();
  if (S > 1) cluster_sync();
  else __syncthreads();

  // ------------------------------------------------------------ join and epilogue
  // token t belongs to rank t % S, a warp per token, four rows per lane
  if (live) {
    const uint32_t mine = sbase + lane * 16;
    auto sum = [&](int row) {
      float4 v = few_ld_cluster(few_mapa(mine + row * FEW_PITCH * 4, 0));
      for (uint32_t s = 1; s < S; ++s) {
        const float4 w = few_ld_cluster(few_mapa(mine + row * FEW_PITCH * 4, s));
        v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
      }
      return v;
    };
    for (int t = (int)rank + warp * (int)S; t < p.T; t += (int)S * (few_threads(MODE) / 32)) {
      if constexpr (MODE == GATE_UP) {
        if (!flag[t]) continue;
        float v[4];
        const float w = wsel[t];
        const float4 g = sum(t), u = sum(p.NT + t);
        const float gg[4] = {g.x, g.y, g.z, g.w}, uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = __fmul_rn(w, __fmul_rn(__fdiv_rn(gg[i], __fadd_rn(1.f, expf(-gg[i]))), uu[i]));
        // channels 4 lane .. 4 lane + 3: strides 1 and 2 here, 4 .. across lanes
        float a = v[0], b = v[2];
        v[0] = __fadd_rn(a, v[1]); v[1] = __fsub_rn(a, v[1]);
        v[2] = __fadd_rn(b, v[3]); v[3] = __fsub_rn(b, v[3]);
        a = v[0]; b = v[1];
        v[0] = __fadd_rn(a, v[2]); v[2] = __fsub_rn(a, v[2]);
        v[1] = __fadd_rn(b, v[3]); v[3] = __fsub_rn(b, v[3]);
        for (int m = 1; m < p.block2 / 4; m <<= 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, v[i], m);
            v[i] = lane & m ? __fsub_rn(o, v[i]) : __fadd_rn(v[i], o);
          }
        }
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = __fmul_rn(v[i], p.inv_sqrt_b2);
          am = fmax_nan(am, fabsf(v[i]));
        }
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) am = fmax_nan(am, __shfl_xor_sync(0xffffffffu, am, m));
        const uint32_t sb = mx_scale_byte(am);
        const float inv = mx_inv_scale(sb);
        const uint32_t lo = cvt_e2m1x2(__fmul_rn(v[1], inv), __fmul_rn(v[0], inv));
        const uint32_t hi = cvt_e2m1x2(__fmul_rn(v[3], inv), __fmul_rn(v[2], inv));
        const size_t row = (size_t)blockIdx.y * p.T + t;
        reinterpret_cast<uint16_t*>(p.hq)[(row * (p.N / 2) + n0 / 2) / 2 + lane] =
            sb == 255u ? (uint16_t)0 : (uint16_t)(lo | hi << 8);
        if ((lane & 7) == 0)
          p.hq_sf[(size_t)blockIdx.y * (p.N / 128) * 512 + mx_sf_offset(t, n0 / 32 + lane / 8, p.N)] = (uint8_t)sb;
      } else {
        float4 y = sum(t);
        float v[4] = {y.x, y.y, y.z, y.w};
        const int nn = n0 + 4 * lane;
        if constexpr (MODE == LINEAR) {
          if (p.c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float s = 0.f;
              if (nn + i < p.N)
                for (int j = 0; j < p.r; ++j)
                  s = fmaf(bf16_bits_to_f32(p.c[(size_t)t * p.r + j]), bf16_bits_to_f32(p.L[(size_t)(nn + i) * p.r + j]), s);
              v[i] += s;
            }
          }
        }
        const size_t at = (size_t)t * p.N + nn;
        if (p.out_fp32) {
          float* out = static_cast<float*>(p.Y) + at;
          if (nn + 4 <= p.N && (p.N & 3) == 0) {
            *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (nn + i < p.N) out[i] = v[i];
          }
        } else {
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.Y) + at;
          if (nn + 4 <= p.N && (p.N & 3) == 0) {
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(v[0], v[1]), b1 = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2*>(out) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (nn + i < p.N) out[i] = __float2bfloat16_rn(v[i]);
          }
        }
      }
    }
  }
  // the partial sums stay until every rank has read them
  if (S > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// ------------------------------------------------------------------ host side
// Ranks per cluster: as many as keep the grid within `fill` CTAs, two steps each at
// least.  33 tiles of 32 steps: 12.7, 9.9, 8.4, 9.1 us with 1, 2, 4, 8 ranks.
int few_ranks(int64_t clusters, int steps, int fill) {
  int S = 1;
  while (S < 8 && clusters * 2 * S <= fill && 4 * S <= steps) S *= 2;
  return S;
}

// `tiles` x `ny` clusters, `steps` K steps to split.
template <int MODE>
cudaError_t launch_mode(const FewMaps& tm, FewParams p, int tiles, int ny, int steps, int sms, cudaStream_t st) {
  constexpr int NA = MODE == GATE_UP ? 2 : 1;
  static SmemLimit limit_once;
  cudaError_t e = limit_once.raise(reinterpret_cast<const void*>(mx_few_kernel<MODE>));
  if (e != cudaSuccess) return e;
  // An SM for every CTA (FUSED: half an SM).  The gate/up products split only while
  // half the SMs are left, where the down products' CTAs start and fetch their
  // weights early (64 tiles: 19.6 us for the layer with 1 rank, 21.2 with 2).
  const int fill = MODE == GATE_UP ? sms / 2 : MODE == FUSED ? 2 * sms : sms;
  int S = few_ranks((int64_t)tiles * ny, steps, fill);
  const int stage = NA * (128 * 128 + 1024) + (MODE == FUSED ? 0 : p.NT * 128 + 1024);
  const int parts = (NA * p.NT * FEW_PITCH * 4 + 1023) & ~1023;   // the partial sums overlay the stages
  int x_bytes = 0, rows_bytes = 0;   // FUSED: the token codes and scales of every step, the rows, the table's entries
  int rot_bytes = 0, most;
  for (;; S /= 2) {
    most = (steps + S - 1) / S;
    if constexpr (MODE == FUSED) {
      const int U = p.block < 64 ? 64 : p.block;
      x_bytes = (most * (p.NT * 128 + FUSED_SF) + 256 + 1023) & ~1023;
      rows_bytes = (p.T * p.K * 2 + 1023) & ~1023;
      rot_bytes = ((most * 256 + 2 * U) * 4 + 1023) & ~1023;
    }
    // one CTA per SM, shared memory full of stages, if all are resident that way (a
    // cluster's CTAs lie in one group of SMs: 148, 148, 132 and 120 for clusters of
    // 1, 2, 4 and 8 on 148 SMs); otherwise two share an SM
    const int64_t room = S <= 2 ? sms : S == 4 ? sms * 8 / 9 : sms * 4 / 5;
    const int limit = (int64_t)tiles * ny * S > room ? 115712 : 230400;
    p.stages = (limit - FEW_TAIL - 1024 - x_bytes - rows_bytes - rot_bytes) / stage;
    // FUSED: beside long rows half an SM has room for few stages or none; fewer
    // ranks with a whole SM each then (us with two stages in half an SM, and this way:
    // 1 x 6144 x 14336, blocks of 1024: 17.5, 14.9; 4 x 4096 x 12288: 16.8, 16.0; with one
    // stage, 2 x 8192 x 18900, blocks of 512: 29.9, 24.2; with three half an SM is as good
    // or better: 3 x 4096 x 14336: 14.2, 14.5; 2 x 5120 x 11008: 13.9, 14.5)
    if (MODE != FUSED || S == 1 || p.stages >= FUSED_MIN_STAGES) break;
  }
  if (p.stages < 1) return cudaErrorInvalidValue;
  if (p.stages > FEW_MAX_STAGES) p.stages = FEW_MAX_STAGES;
  if (p.stages > most) p.stages = most < 1 ? 1 : most;
  p.off_x = p.stages * stage > parts ? p.stages * stage : parts;
  p.off_rows = p.off_x + x_bytes;
  p.off_rot = p.off_rows + rows_bytes;
  p.tail = p.off_rot + rot_bytes;
  uint32_t cols = 32;
  while ((int)cols < NA * p.NT + p.stages * (NA + 1) * 8) cols *= 2;
  p.tmem_cols = cols;
  // shared memory is taken in at least the proportion of TMEM (of 228 KB, 1 KB
  // of it the system's per CTA): CTAs that share an SM by the one fit by the
  // other, so that no allocation waits for a CTA that waits for its cluster
  int smem = p.tail + FEW_TAIL + 1024;
  const int share = (int)cols * 456 - 1024;
  if (smem < share) smem = share;
  // nor, in a cluster, for a neighbour that takes all of TMEM and half of shared memory
  if (S > 1 && smem < 115712) smem = 115712;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * S), (unsigned)ny);
  cfg.blockDim = dim3(few_threads(MODE));
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, mx_few_kernel<MODE>, tm, p);
}

int token_columns(int T) { return (T + 15) / 16 * 16; }

}  // namespace

// With the low-rank branch the epilogue reads r values of L for each of a rank's
// tokens, one after another: about r (4 + tokens per rank), as against the longer
// way of the one-CTA kernel of rq_k2.cu (128 x 128 tiles, no split of K) through K,
// about K / 32 in the same unit.  us here and there: 64 x 4096 x 12288, r = 32: 153.6
// and 12.4; r = 8: 29.0 and 12.5, for 8 tokens 11.9 and 12.7; 4096 outputs of 16384
// columns, r = 32, 32 and 64 tokens: 29.9 and 31.0, 48.7 and 31.1; of 8192 columns, 8 and
// 16 tokens: 15.8 and 17.8, 19.5 and 17.8; 1 x 1152 x 1152, r = 8: 5.7 and 5.5.
bool mx_few_low_rank(int M, int N, int K, int r, int sms) {
  const int S = few_ranks((N + 127) / 128, (K + 255) / 256, sms > 0 ? sms : 148);
  return r * (4 + (M + S - 1) / S) * 32 < K;
}

cudaError_t launch_mx_few(const GemmLaunch& a, cudaStream_t st, const char** why) {
  FewMaps tm;
  FewParams p{};
  p.T = a.M; p.NT = token_columns(a.M); p.K = a.K; p.N = a.N;
  p.early = a.early_weights;
  p.w_sf = a.w_bscale; p.x_sf = a.a_bscale;
  p.c = a.c; p.L = a.L; p.r = a.r;
  p.Y = a.Y; p.out_fp32 = a.out_fp32;
  p.status = a.status; p.wait_ns = a.wait_ns; p.inject_tx = a.inject_tx;
  if (!mx_code_map(&tm.w, a.w_codes, a.N, a.K, 128) || !mx_code_map(&tm.x, a.a_codes, a.M, a.K, p.NT)) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  return launch_mode<LINEAR>(tm, p, (a.N + 127) / 128, 1, (a.K + 255) / 256, a.num_sms > 0 ? a.num_sms : 148, st);
}

// The rows of a few tokens fit beside the weights' stages, and there is an SM for
// every tile of 128 outputs, so that a plan with one rank and a whole SM each always
// exists; the redundant transform is a few thousand values per CTA.  Two CTAs of 384
// threads per SM leave 80 registers, of which the transform's loops spill 60 bytes.
bool mx_layer_fused(int M, int N, int K, int sms) {
  return M <= 4 && (int64_t)M * K <= 16384 && K <= 8192 && (N + 127) / 128 <= sms;
}

cudaError_t launch_mx_layer_fused(const GemmLaunch& a, const uint16_t* x, const int32_t* rot, int block, float inv_sqrt_b,
                                  cudaStream_t st) {
  FewMaps tm;
  FewParams p{};
  p.T = a.M; p.NT = token_columns(a.M); p.K = a.K; p.N = a.N;
  p.w_sf = a.w_bscale;
  p.xb = x; p.rot = rot; p.block = block; p.inv_sqrt_b = inv_sqrt_b;
  p.Y = a.Y; p.out_fp32 = a.out_fp32;
  p.status = a.status; p.wait_ns = a.wait_ns; p.inject_tx = a.inject_tx;
  if (!mx_code_map(&tm.w, a.w_codes, a.N, a.K, 128)) return cudaErrorInvalidValue;
  tm.x = tm.w;   // (not used)
  return launch_mode<FUSED>(tm, p, (a.N + 127) / 128, 1, (a.K + 255) / 256, a.num_sms > 0 ? a.num_sms : 148, st);
}

cudaError_t launch_moe_products(const MoeLaunch& a, const uint8_t* xq, const uint8_t* xq_sf, uint8_t* hq, uint8_t* hq_sf,
                                int active, cudaStream_t st) {
  const int sms = a.num_sms > 0 ? a.num_sms : 148;
  FewMaps tm;
  FewParams p{};
  p.T = a.T; p.NT = token_columns(a.T); p.K = a.K; p.N = a.I;
  p.w_sf = a.w1_sf; p.w_sf_expert = mx_sf_bytes(2 * a.I, a.K);
  p.x_sf = xq_sf;
  p.idx = a.idx; p.wts = a.wts; p.top_k = a.top_k;
  p.hq = hq; p.hq_sf = hq_sf; p.block2 = a.block2; p.inv_sqrt_b2 = a.inv_sqrt_b2;
  p.status = a.status; p.wait_ns = a.wait_ns; p.inject_tx = a.inject_tx;
  if (!mx_code_map(&tm.w, a.w1, (uint64_t)a.E * 2 * a.I, a.K, 128) || !mx_code_map(&tm.x, xq, a.T, a.K, p.NT))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_mode<GATE_UP>(tm, p, a.I / 128, active, (a.K + 255) / 256, sms, st);
  if (e != cudaSuccess) return e;
  p.K = a.I; p.N = a.K;
  p.early = 1;   // the routing was complete before the gate/up kernel let this one start
  p.w_sf = a.w2_sf; p.w_sf_expert = mx_sf_bytes(a.K, a.I);
  p.x_sf = hq_sf;
  p.Y = a.Y; p.out_fp32 = a.out_fp32;
  if (!mx_code_map(&tm.w, a.w2, (uint64_t)a.E * a.K, a.I, 128) ||
      !mx_code_map(&tm.x, hq, (uint64_t)active * a.T, a.I, p.NT))
    return cudaErrorInvalidValue;
  return launch_mode<DOWN>(tm, p, (a.K + 127) / 128, 1, active * ((a.I + 255) / 256), sms, st);
}

}  // namespace rq
