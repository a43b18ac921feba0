// MXFP4: the activation (and weight-row) transform, rotate -> quantize -> pack,
// and codes read back as values.
//
// MXFP4 has no row scale: a block of 32 rotated coordinates is quantized from
// its own maximum, so one pass over the transformed values in registers is
// all there is, and no thread waits for a row's other blocks.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rq_internal.h"
#include "rq_mx.cuh"
#include "rq_ptx.cuh"

namespace rq {

namespace {

// ------------------------------------------------------------ rotate + quantize
// Persistent over groups of R rows (1, 2, 4 or 8), nbuf groups in flight: a group's
// rows land in shared memory by bulk copies, at a pitch that puts the R rows
// 128 / R bytes apart modulo the banks.  A warp's lanes are R rows x 32 / R
// segments of 64 rotated coordinates (a unit); a thread gathers its segment through
// the signed-permutation table (16 bits per coordinate: byte offset, sign in bit
// 15), two chunks of 32 that are one MXFP4 block each.  Units are dealt to the
// warps round robin through the groups, without a barrier between them; the
// last warp to leave a group refills its buffer.
// Butterflies: strides 1 .. 16 inside the chunks, 32 between the two chunks,
// 64 between the chunks after one of them was exchanged with the neighbouring
// segment's (half the shuffles of a butterfly across lanes), 128 and up across
// lanes.  For the exchange the odd segment holds its chunks in reverse, so that
// every lane sends and receives its second chunk; the signs that this turns
// round are +-1 factors of the packed multiply-adds, exact.
// Bound by its instructions: 18 a value, a third of them the gather (mask, add,
// load, shift, sign), at 16 warps of 128 registers.  65520 x 1536: 82 us, 3.1 TB/s
// of the bytes read and written; 4608 x 12288, blocks of 256: 51 us, 2.8 TB/s.  20
// and 24 warps of 96 and 80 registers: 97 and 105 us, 12 and 8: 89 and 90, at the first.
constexpr int MXQ_THREADS = 512;

struct MxqParams {
  const uint16_t* x;
  const int32_t* rot;
  uint8_t* codes;
  uint8_t* sf;
  int32_t* status;
  uint64_t wait_ns;
  uint32_t inject_tx;
  int rows, K, block, lr;   // lr: log2 of the rows per group
  int ngroups, nbuf;
  float isb;                // fp32(1 / sqrt(block))
};

constexpr int MXQ_MAXBUF = 8;
constexpr int MXQ_SEG = 144;   // bytes of a segment's table entries: 64 x 2, and 16 that shift the banks

// (p, q) of two values each -> (s p + q, p - s q), s = +-1
__device__ __forceinline__ void cross2(float& p0, float& p1, float& q0, float& q1, float s) {
  asm("{\n\t.reg .b64 p, q, s, n, a;\n\t"
      "mov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\tmov.b64 n, {%5, %5};\n\t"
      "fma.rn.f32x2 a, s, p, q;\n\tfma.rn.f32x2 q, n, q, p;\n\t"
      "mov.b64 {%0, %1}, a;\n\tmov.b64 {%2, %3}, q;\n\t}"
      : "+f"(p0), "+f"(p1), "+f"(q0), "+f"(q1)
      : "f"(s), "f"(-s));
}
__device__ __forceinline__ void bfly2(float& a0, float& a1, float& b0, float& b1) {
  asm("{\n\t.reg .b64 a, b, s, d;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 s, a, b;\n\tsub.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, s;\n\tmov.b64 {%2, %3}, d;\n\t}"
      : "+f"(a0), "+f"(a1), "+f"(b0), "+f"(b1));
}
// v = s v + o on two values, s = +-1
__device__ __forceinline__ void sfma2(float& v0, float& v1, float s, float o0, float o1) {
  asm("{\n\t.reg .b64 v, o, s;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 o, {%3, %4};\n\tmov.b64 s, {%2, %2};\n\t"
      "fma.rn.f32x2 v, s, v, o;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(v0), "+f"(v1)
      : "f"(s), "f"(o0), "f"(o1));
}
__device__ __forceinline__ void mul2(float& v0, float& v1, float s) {
  asm("{\n\t.reg .b64 v, s;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\t"
      "mul.rn.f32x2 v, v, s;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(v0), "+f"(v1)
      : "f"(s));
}
// max(|a|, |b|, |c|), NaN if one is
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// eight values to eight E2M1 nibbles, the first in the low bits
__device__ __forceinline__ uint32_t pack8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// 32 coordinates of one chunk through the table
__device__ __forceinline__ void gather32(float (&v)[32], const uint8_t* row, const uint8_t* tab) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 t = *reinterpret_cast<const uint4*>(tab + 16 * j);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = w[i], b = w[i] >> 16;
      const uint32_t xa = *reinterpret_cast<const uint16_t*>(row + (a & 0x7FFEu));
      const uint32_t xb = *reinterpret_cast<const uint16_t*>(row + (b & 0x7FFEu));
      v[8 * j + 2 * i] = __uint_as_float((xa ^ (a & 0x8000u)) << 16);
      v[8 * j + 2 * i + 1] = __uint_as_float((xb << 16) ^ (w[i] & 0x80000000u));
    }
  }
}

__device__ __forceinline__ void fwht_chunk(float (&v)[32], int block) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float a = v[e], b = v[e + 1];
    v[e] = __fadd_rn(a, b);
    v[e + 1] = __fsub_rn(a, b);
  }
#pragma unroll
  for (int h = 2; h <= 8; h <<= 1) {
#pragma unroll
    for (int e = 0; e < 32; e += 2)
      if ((e & h) == 0) bfly2(v[e], v[e + 1], v[e + h], v[e + h + 1]);
  }
  if (block > 16) {
#pragma unroll
    for (int e = 0; e < 16; e += 2) bfly2(v[e], v[e + 1], v[e + 16], v[e + 17]);
  }
}

// Scale byte and packed codes of a transformed chunk (before the 1/sqrt(block)).
// Rounding is monotone, so the largest |y| is that of the largest |v|.  One
// product by isb 2^(127 - byte) then equals the two roundings of the stated
// order, (v isb) rounded and scaled exactly, unless something is subnormal:
// at byte 32 a subnormal y lands below 2^-31 and is 0 either way, and the
// factor itself is normal up to byte 240; outside both steps are taken.
__device__ __forceinline__ uint32_t quantize32(float (&v)[32], float isb, uint4& out) {
  float am = fabsf(v[0]);
#pragma unroll
  for (int e = 1; e < 31; e += 2) am = max3_abs(am, v[e], v[e + 1]);
  am = max3_abs(am, v[31], 0.f);
  const uint32_t sb = mx_scale_byte(__fmul_rn(am, isb));
  float f = mx_inv_scale(sb);
  if (sb < 32u || sb > 240u) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) mul2(v[e], v[e + 1], isb);
  } else {
    f *= isb;
  }
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) mul2(v[8 * j + e], v[8 * j + e + 1], f);
    w[j] = sb == 255u ? 0u : pack8(v + 8 * j);
  }
  out = make_uint4(w[0], w[1], w[2], w[3]);
  return sb;
}

__global__ void __launch_bounds__(MXQ_THREADS, 1) mx_quantize_kernel(const __grid_constant__ MxqParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int K = p.K, lr = p.lr, R = 1 << lr;
  const int nseg = K / 64;
  const int pitch = 2 * K + (lr ? 128 >> lr : 0);
  uint8_t* tab = smem;
  uint8_t* rowbuf = smem + nseg * MXQ_SEG;              // [nbuf][R][pitch]
  uint64_t* full = reinterpret_cast<uint64_t*>(rowbuf + p.nbuf * R * pitch);
  int* done = reinterpret_cast<int*>(full + MXQ_MAXBUF);   // warps that have left a buffer's group
  int* fills = done + MXQ_MAXBUF;                          // groups that went into a buffer so far
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(fills + MXQ_MAXBUF);
  const int nthreads = blockDim.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = nthreads >> 5;
  const int mine = ((int)p.ngroups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;   // this CTA's groups

  auto issue = [&](int j) {   // this CTA's j-th group, into buffer j % nbuf
    const int buf = j % p.nbuf, r0 = ((int)blockIdx.x + j * (int)gridDim.x) << lr, nr = min(R, p.rows - r0);
    ++fills[buf];
    mbar_expect_tx(&full[buf], (uint32_t)nr * 2 * K + (j == 0 ? p.inject_tx : 0u));
    for (int i = 0; i < nr; ++i)
      bulk_g2s(rowbuf + (buf * R + i) * pitch, p.x + (size_t)(r0 + i) * K, (uint32_t)(2 * K), &full[buf]);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.nbuf; ++i) {
      mbar_init(&full[i], 1);
      done[i] = fills[i] = 0;
    }
    *abort_flag = 0;
    fence_mbar_init();
    for (int j = 0; j < min(mine, p.nbuf); ++j) issue(j);
    // the product that reads these codes may be scheduled: it waits for this
    // grid before it reads them
    griddep_launch_dependents();
  }
  for (int i = threadIdx.x; i < K / 4; i += nthreads) {
    const int4 r = __ldg(reinterpret_cast<const int4*>(p.rot) + i);
    auto entry = [](int32_t v) { return (uint32_t)(v & 0x3FFF) << 1 | (v < 0 ? 0x8000u : 0u); };
    *reinterpret_cast<uint2*>(tab + (i / 16) * MXQ_SEG + (i % 16) * 8) =
        make_uint2(entry(r.x) | entry(r.y) << 16, entry(r.z) | entry(r.w) << 16);
  }
  __syncthreads();

  const int spw = 32 >> lr;                              // segments per warp
  const int rl = lane & (R - 1), sl = lane >> lr;
  const int nunits = (nseg + spw - 1) / spw;
  // Every warp walks through all groups in order, also one without a unit there:
  // its answer from a buffer's barrier is then always that of the next phase.
  int first = warp;   // this warp's first unit of the group
  int buf = 0, ph = 0;
  for (int j = 0; j < mine; ++j) {
    if (!warp_wait(&full[buf], ph, p.status, ST_TIMEOUT_LOAD, abort_flag, p.wait_ns)) break;
    const int r0 = ((int)blockIdx.x + j * (int)gridDim.x) << lr, nr = min(R, p.rows - r0);
    for (int u = first; u < nunits; u += nwarps) {
      const int seg = u * spw + sl;
      const bool live = seg < nseg && rl < nr;
      const bool odd = p.block > 64 && (seg & 1);
      const uint8_t* t = tab + min(seg, nseg - 1) * MXQ_SEG;
      const uint8_t* row = rowbuf + (buf * R + rl) * pitch;
      float a[32], b[32];
      gather32(a, row, t + (odd ? 64 : 0));
      gather32(b, row, t + (odd ? 0 : 64));
      fwht_chunk(a, p.block);
      fwht_chunk(b, p.block);
      const float s = odd ? -1.f : 1.f;
      if (p.block > 32) {
#pragma unroll
        for (int e = 0; e < 32; e += 2) cross2(a[e], a[e + 1], b[e], b[e + 1], s);
      }
      int ca = seg * 2 + (odd ? 1 : 0), cb = seg * 2 + 1;   // the chunks that a and b hold
      if (p.block > 64) {
#pragma unroll
        for (int e = 0; e < 32; ++e) b[e] = __shfl_xor_sync(0xffffffffu, b[e], R);
#pragma unroll
        for (int e = 0; e < 32; e += 2) cross2(a[e], a[e + 1], b[e], b[e + 1], s);
        cb = odd ? seg * 2 - 1 : seg * 2 + 2;
        for (int m = 2; m * 64 < p.block; m <<= 1) {
          const float sg = seg & m ? -1.f : 1.f;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float o0 = __shfl_xor_sync(0xffffffffu, a[e], m << lr), o1 = __shfl_xor_sync(0xffffffffu, a[e + 1], m << lr);
            sfma2(a[e], a[e + 1], sg, o0, o1);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float o0 = __shfl_xor_sync(0xffffffffu, b[e], m << lr), o1 = __shfl_xor_sync(0xffffffffu, b[e + 1], m << lr);
            sfma2(b[e], b[e + 1], sg, o0, o1);
          }
        }
      }
      uint4 pa, pb;
      const uint32_t sa = quantize32(a, p.isb, pa), sb = quantize32(b, p.isb, pb);
      // the four scale bytes of 128 columns meet in the even segment's lane
      const uint32_t w = sa << (8 * (ca & 3)) | sb << (8 * (cb & 3));
      const uint32_t o = __shfl_xor_sync(0xffffffffu, w, R);
      if (live) {
        uint8_t* dst = p.codes + (size_t)(r0 + rl) * (K / 2);
        *reinterpret_cast<uint4*>(dst + ca * 16) = pa;
        *reinterpret_cast<uint4*>(dst + cb * 16) = pb;
        if (!(seg & 1)) {
          uint8_t* sf = p.sf + mx_sf_offset(r0 + rl, seg * 2, K);
          if (seg + 1 < nseg) *reinterpret_cast<uint32_t*>(sf) = w | o;
          else *reinterpret_cast<uint16_t*>(sf) = (uint16_t)w;   // K an odd multiple of 64
        }
      }
    }
    __syncwarp();
    if (lane == 0) {
      __threadfence_block();
      if (atomicAdd(&done[buf], 1) == nwarps - 1) {
        done[buf] = 0;
        if (j + p.nbuf < mine) {
          fence_proxy_async_smem();
          issue(j + p.nbuf);
        }
      }
    }
    first = (first - nunits) % nwarps;   // the deal goes on where this group ended
    if (first < 0) first += nwarps;
    if (++buf == p.nbuf) { buf = 0; ph ^= 1; }
  }
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0)   // let the copies in flight land (bounded) before the shared memory goes away
    for (int i = 0; i < p.nbuf; ++i)
      if (fills[i]) mbar_drain(&full[i], (fills[i] - 1) & 1, p.wait_ns);
}

// ----------------------------------------------------------------- dequantize
// A thread per block: 16 bytes of codes, a scale byte, 32 values out in whole
// 32-byte sectors; 2^tx threads along a row.  4608 x 12288 to BF16: 24.7 us, 5.8 TB/s
// of the bytes read and written (35 us with 16-byte stores and a thread per 8 codes).
__device__ __forceinline__ void store32(void* dst, const uint32_t* w, bool wide) {
  if (!wide) {   // an output that starts in the middle of a sector
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <typename T>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* codes, const uint8_t* bscale, T* out,
                                                            int rows, int K, int tx) {
  const int blocks = K / 32;
  const int x = threadIdx.x & ((1 << tx) - 1), y = threadIdx.x >> tx, per = 256 >> tx;
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  for (int m = (int)blockIdx.x * per + y; m < rows; m += (int)gridDim.x * per) {
    const uint4* c = reinterpret_cast<const uint4*>(codes + (size_t)m * (K / 2));
    T* o = out + (size_t)m * K;
#pragma unroll 2
    for (int kb = x; kb < blocks; kb += 1 << tx) {
      const uint4 q4 = __ldg(c + kb);
      const float s = mx_scale(__ldg(bscale + mx_sf_offset(m, kb, K)));
      const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
      uint32_t w[32 * sizeof(T) / 4];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        uint32_t h;   // two E2M1 -> two FP16, exact
        asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(q[e / 8] >> (4 * (e & 7))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        if constexpr (sizeof(T) == 4) {
          w[e] = __float_as_uint(f.x * s);
          w[e + 1] = __float_as_uint(f.y * s);
        } else {
          const __nv_bfloat162 b2 = __floats2bfloat162_rn(f.x * s, f.y * s);
          w[e / 2] = *reinterpret_cast<const uint32_t*>(&b2);
        }
      }
#pragma unroll
      for (int i = 0; i < (int)sizeof(T); ++i) store32(reinterpret_cast<uint8_t*>(o + kb * 32) + 32 * i, w + 8 * i, wide);
    }
  }
}

// ------------------------------------------------------------------ tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn find_encode() {
  void* f = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    return reinterpret_cast<EncodeTiledFn>(f);
  return nullptr;
}

bool map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t rows, uint64_t pitch,
            uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  static const EncodeTiledFn enc = find_encode();
  if (!enc) return false;
  cuuint64_t dims[2] = {inner, rows}, strides[1] = {pitch};
  cuuint32_t box[2] = {box_inner, box_rows}, es[2] = {1, 1};
  return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool mx_code_map(CUtensorMap* m, const uint8_t* codes, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  return map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, cols / 2, rows, cols / 2, 128, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool mx_scale_map(CUtensorMap* m, const uint8_t* sf, uint64_t rows, uint64_t cols) {
  return map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, sf, 128, (rows + 127) / 128 * ((cols + 127) / 128), 512, 128, 2,
                CU_TENSOR_MAP_SWIZZLE_NONE);
}
bool mx_out_map(CUtensorMap* m, void* Y, uint64_t rows, uint64_t cols) {
  return map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y, cols, rows, cols * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

cudaError_t launch_mx_quantize(const K1Launch& a, cudaStream_t st) {
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void*>(mx_quantize_kernel));
  if (e != cudaSuccess) return e;
  const int sms = a.num_sms > 0 ? a.num_sms : 148;
  const int table = a.K / 64 * MXQ_SEG;
  auto group = [&](int lr) { return (2 * a.K + (lr ? 128 >> lr : 0)) << lr; };   // bytes of a group's rows
  // rows per group: as many as put their gathers on different banks (8 rows: 2.1
  // expected cycles for 32 lanes, 4 rows: 2.6, one row: 3.5); a Hadamard block has
  // to lie in one warp (32 / R segments of 64), two groups in shared memory, and few
  // rows are spread over the SMs
  int lr = a.block <= 256 ? 3 : a.block == 512 ? 2 : 1;
  while (lr > 0 && (a.rows >> lr) < sms) --lr;
  while (lr > 0 && table + 2 * group(lr) > 232000) --lr;
  MxqParams p{};
  p.x = a.x; p.rot = a.rot; p.codes = a.codes; p.sf = a.bscale;
  p.status = a.status; p.wait_ns = a.wait_ns; p.inject_tx = a.inject_tx;
  p.rows = a.rows; p.K = a.K; p.block = a.block; p.lr = lr; p.isb = a.inv_sqrt_b;
  p.ngroups = (a.rows + (1 << lr) - 1) >> lr;
  const int units = (a.K / 64 + (32 >> lr) - 1) / (32 >> lr);
  // two CTAs of 8 warps per SM if three groups fit half of its shared memory, else
  // one of 16; fewer warps when the CTA has fewer units
  const bool two = table + 3 * group(lr) <= 115000;
  const int room = (two ? 115000 : 232000) - table;
  p.nbuf = room / group(lr) < MXQ_MAXBUF ? room / group(lr) : MXQ_MAXBUF;
  const int most = sms * (two ? 2 : 1), grid = p.ngroups < most ? p.ngroups : most;
  const int turns = (p.ngroups + grid - 1) / grid;
  if (p.nbuf > turns) p.nbuf = turns;
  const int64_t all = (int64_t)units * turns;
  // (warps without a unit help with the table)
  const int want = all > 4 ? (int)(all < 16 ? all : 16) : 4, cap = two ? 8 : 16;
  const int warps = want < cap ? want : cap;
  const int smem = table + p.nbuf * group(lr) + MXQ_MAXBUF * 16 + 16;
  mx_quantize_kernel<<<grid, warps * 32, smem, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_mx_dequantize(const MxDequantLaunch& a, cudaStream_t st) {
  int tx = 1;   // the threads along a row: a power of two up to 256, at most its blocks
  while (tx < 8 && (2 << tx) <= a.K / 32) ++tx;
  const int per = 256 >> tx;
  const int64_t blocks = ((int64_t)a.rows + per - 1) / per, most = (int64_t)(a.num_sms > 0 ? a.num_sms : 148) * 32;
  const int grid = (int)(blocks < most ? blocks : most);
  if (a.out_fp32)
    mx_dequantize_kernel<float><<<grid, 256, 0, st>>>(a.codes, a.bscale, static_cast<float*>(a.out), a.rows, a.K, tx);
  else
    mx_dequantize_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a.codes, a.bscale, static_cast<__nv_bfloat16*>(a.out), a.rows, a.K, tx);
  return cudaGetLastError();
}

}  // namespace rq
