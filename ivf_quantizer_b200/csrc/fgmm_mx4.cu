// 4-bit codes of vectors (OCP Microscaling Formats v1.0, MXFP4: blocks of 32 e2m1 codes with
// one e8m0 scale) and the scores of queries against them.  The layout of codes and scales is
// that of include/fgmm.h.
//
//   encode  reads 4 (or 2) bytes a value, writes 17/32: bound by reading
//   decode  the reverse: bound by writing
//   scores  out = alpha Q X^T + bias over the decoded values
#include <cuda_bf16.h>

#include "fgmm_internal.h"
#include "sm100_ptx.cuh"

namespace fgmm {
namespace {

constexpr int kMxThreads = 256;

__device__ __forceinline__ float mx_ld(const float* p) { return __ldg(p); }
__device__ __forceinline__ float mx_ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void mx_ld4(const float* p, float (&v)[4]) {
  const float4 t = __ldcs(reinterpret_cast<const float4*>(p));
  v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
}
__device__ __forceinline__ void mx_ld4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 t = __ldcs(reinterpret_cast<const uint2*>(p));
  v[0] = __uint_as_float(t.x << 16), v[1] = __uint_as_float(t.x & 0xffff0000u);
  v[2] = __uint_as_float(t.y << 16), v[3] = __uint_as_float(t.y & 0xffff0000u);
}
__device__ __forceinline__ void mx_st(float* p, float v) { *p = v; }
__device__ __forceinline__ void mx_st(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void mx_st4(float* p, const float (&v)[4]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
}
__device__ __forceinline__ void mx_st4(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  uint2 t;
  t.x = reinterpret_cast<const uint32_t&>(a);
  t.y = reinterpret_cast<const uint32_t&>(b);
  __stcs(reinterpret_cast<uint2*>(p), t);
}

// Four values, already scaled, to four e2m1 codes (nearest, ties to even, saturating).
__device__ __forceinline__ uint32_t mx_codes4(const float (&v)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b, a, b};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
  return r & 0xffffu;
}
// Four e2m1 codes (the low 16 bits) to their values.  The three magnitude bits (two of exponent,
// bias 1, one of mantissa) placed at the top of a float's mantissa and the bottom of its exponent
// read as the value times 2^-126, the subnormal 0.5 included.
__device__ __forceinline__ void mx_values4(uint32_t c, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = c >> (4 * j);
    v[j] = __uint_as_float((b & 7u) << 22 | (b & 8u) << 28) * 8.507059173023462e37f;  // 2^126
  }
}
// The value of an e8m0 scale byte.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return s == 255u ? __int_as_float(0x7fc00000)
                   : (s == 0u ? __int_as_float(0x00400000) : __int_as_float((int)(s << 23)));
}

// One warp encodes 128 dimensions (four blocks) of the rows r, r + 32, r + 64, r + 96 of a
// 128-row tile: four dimensions a lane, eight lanes a block.  Four independent loads a lane are
// in flight, a row's 128 values are one contiguous read, and the sixteen scales are the 16
// contiguous bytes that the scale tile gives these rows.  VEC: rows allow 4-value loads.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMxThreads)
    mx4_encode_kernel(const T* __restrict__ X, int64_t n, int D, int64_t ldx, int nb, int nkc,
                      int64_t groups, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (kMxThreads / 32);
  for (int64_t g = (int64_t)blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5); g < groups;
       g += step) {
    const int64_t rr = g / nkc;                 // row tile * 32 + row within the quarter
    const int kc = (int)(g - rr * nkc);
    const int64_t row0 = (rr >> 5) * 128 + (rr & 31);
    const int d = kc * 128 + lane * 4;
    float v[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t row = row0 + 32 * c;
      const T* p = X + row * ldx + d;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[c][j] = 0.f;
      if (row < n) {
        if (VEC && d + 4 <= D) {
          mx_ld4(p, v[c]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (d + j < D) v[c][j] = mx_ld(p + j);
        }
      }
    }
    uint32_t words[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // magnitudes as integers: NaN and infinity sort above every finite value
      uint32_t a = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) a = max(a, __float_as_uint(v[c][j]) & 0x7fffffffu);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
      const uint32_t e = a >> 23;
      uint32_t s = e > 2u ? e - 2u : 0u;        // floor(log2 a) - 2 + 127, at least 0
      const float inv = __uint_as_float((254u - s) << 23);
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = v[c][j] * inv;
      uint32_t code = mx_codes4(y);
      if (e == 255u) s = 255u, code = 0u;
      const int64_t row = row0 + 32 * c;
      if (row < n && d < nb * 32)
        *reinterpret_cast<uint16_t*>(codes + row * ((int64_t)nb * 16) + (d >> 1)) = (uint16_t)code;
      uint32_t w = s << (8 * (lane >> 3));
      w |= __shfl_xor_sync(0xffffffffu, w, 8);
      w |= __shfl_xor_sync(0xffffffffu, w, 16);
      words[c] = w;
    }
    if (lane == 0)
      *reinterpret_cast<uint4*>(scales + ((rr >> 5) * nkc + kc) * 512 + (rr & 31) * 16) =
          make_uint4(words[0], words[1], words[2], words[3]);
  }
}

// The same assignment of rows and dimensions to warps and lanes as in mx4_encode_kernel.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMxThreads)
    mx4_decode_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      int64_t n, int D, int nb, int nkc, int64_t groups, T* __restrict__ out,
                      int64_t ldo) {
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * (kMxThreads / 32);
  for (int64_t g = (int64_t)blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5); g < groups;
       g += step) {
    const int64_t rr = g / nkc;
    const int kc = (int)(g - rr * nkc);
    const int64_t row0 = (rr >> 5) * 128 + (rr & 31);
    const int d = kc * 128 + lane * 4;
    const uint4 sw = __ldg(reinterpret_cast<const uint4*>(
        scales + ((rr >> 5) * nkc + kc) * 512 + (rr & 31) * 16));
    const uint32_t words[4] = {sw.x, sw.y, sw.z, sw.w};
    uint32_t code[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t row = row0 + 32 * c;
      code[c] = (row < n && d < D) ? __ldcs(reinterpret_cast<const uint16_t*>(
                                         codes + row * ((int64_t)nb * 16) + (d >> 1)))
                                   : 0u;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t row = row0 + 32 * c;
      if (row >= n) continue;
      const float s = mx_scale((words[c] >> (8 * (lane >> 3))) & 255u);
      float v[4];
      mx_values4(code[c], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= s;
      T* p = out + row * ldo + d;
      if (VEC && d + 4 <= D) {
        mx_st4(p, v);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (d + j < D) mx_st(p + j, v[j]);
      }
    }
  }
}

// ------------------------------------------------------------------ scores (tcgen05)
// The vectors are the M side of the products (128 of them a tile: TMEM lane = vector), the
// queries the N side (NT a tile: TMEM column = query).  The codes then stream through the wide
// side whatever the number of queries, and a warp's 32 lanes write 32 consecutive scores of one
// query: whole 128-byte lines from registers, for any N and any row stride.
//
// One CTA a SM walks its tiles: a TMA warp fills a ring of stages (256 dimensions of 128 vectors
// and NT queries, 128 bytes a row, and their scale tiles), one thread copies a stage's scales to
// TMEM and issues its four K = 64 block-scaled products, and the epilogue warps drain one of two
// accumulators while the other is filled.
constexpr int kMxBM = 128;         // vectors a tile
constexpr int kMxRowB = 128;       // bytes of a row in a stage: 256 dimensions
constexpr int kMxSfB = 1024;       // scale bytes of 128 rows in a stage: two tiles of 512

template <int NT>
struct MxCfg {
  static constexpr int kStage = kMxBM * kMxRowB + NT * kMxRowB + 2 * kMxSfB;
  static constexpr int kStages = (216 * 1024) / kStage < 10 ? (216 * 1024) / kStage : 10;
  static constexpr int kEpiWarps = NT >= 64 ? 8 : 4;
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kCols = NT == 128 ? 512 : 4 * NT < 64 ? 64 : 4 * NT;  // TMEM columns
  static constexpr int kSfCol = 2 * NT;             // two scale sets of 16 columns behind the sums
};

struct MxBars {
  uint64_t full[10], empty[10], s_full[2], s_empty[2], drain;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ void mx_timeout(int* status, MxBars* bars) {
  if (status) atomicCAS(status, FGMM_OK, FGMM_ERR_TIMEOUT);
  bars->abort = 1;
}

template <int NT, typename T>
__global__ void __launch_bounds__(MxCfg<NT>::kThreads, 1)
    mx4_scores_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmq,
                      const uint8_t* __restrict__ xs, const uint8_t* __restrict__ qs, int64_t n,
                      int64_t m, int nb, int64_t ntiles, int mtiles, float alpha,
                      const float* __restrict__ bias, T* __restrict__ out, int64_t ldo, int* status) {
  using C = MxCfg<NT>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  MxBars* bars = reinterpret_cast<MxBars*>(ring + C::kStages * C::kStage);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nkc = (nb + 3) / 4;                     // scale tiles (128 dimensions) of a row
  const int nst = (nkc + 1) / 2;                    // stages of a tile
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&bars->full[s], 1);
      ptx::mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&bars->s_full[b], 1);
      ptx::mbar_init(&bars->s_empty[b], C::kEpiWarps);
    }
    ptx::mbar_init(&bars->drain, 1);
    bars->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&bars->tmem, C::kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem;

  if (warp == 0) {
    if (lane == 0) {
      ptx::prefetch_tmap(&tmx);
      ptx::prefetch_tmap(&tmq);
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < ntiles && !*abort; t += gridDim.x) {
        const int64_t nt = t / mtiles;
        const int mt = (int)(t - nt * mtiles);
        for (int k = 0; k < nst; ++k, ++it) {
          const int s = it % C::kStages;
          if (it >= C::kStages && !ptx::mbar_wait(&bars->empty[s], ((it / C::kStages) - 1) & 1, abort)) {
            mx_timeout(status, bars);
            ok = false;
            break;
          }
          unsigned char* a = ring + s * C::kStage;
          unsigned char* b = a + kMxBM * kMxRowB;
          unsigned char* sf = b + NT * kMxRowB;
          const uint32_t sfb = (nkc - 2 * k >= 2 ? 2 : 1) * 512;
          ptx::mbar_arrive_expect_tx(&bars->full[s], kMxBM * kMxRowB + NT * kMxRowB + 2 * sfb);
          ptx::tma_load_2d(a, &tmx, &bars->full[s], k * kMxRowB, (int)(nt * kMxBM));
          ptx::bulk_load(sf, xs + (nt * nkc + 2 * k) * 512, sfb, &bars->full[s]);
          ptx::tma_load_2d(b, &tmq, &bars->full[s], k * kMxRowB, mt * NT);
          ptx::bulk_load(sf + kMxSfB, qs + ((int64_t)mt * nkc + 2 * k) * 512, sfb, &bars->full[s]);
        }
      }
      if (*abort)  // let every copy this thread started land before the CTA exits
        for (uint32_t k = (it > C::kStages ? it - C::kStages : 0); k < it; ++k)
          ptx::mbar_drain(&bars->full[k % C::kStages], (k / C::kStages) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint64_t kHiK = ptx::sw128_hi(16, 1024);
      uint32_t it = 0, j = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < ntiles && !*abort; t += gridDim.x, ++j) {
        const uint32_t buf = j & 1;
        if (j >= 2 && !ptx::mbar_wait(&bars->s_empty[buf], ((j >> 1) - 1) & 1, abort)) {
          ok = false;
          break;
        }
        const uint32_t d_tmem = tmem + buf * NT;
        for (int k = 0; k < nst; ++k, ++it) {
          const int s = it % C::kStages;
          if (!ptx::mbar_wait(&bars->full[s], (it / C::kStages) & 1, abort)) {
            ok = false;
            break;
          }
          const uint32_t a = ptx::smem_u32(ring + s * C::kStage);
          const uint32_t b = a + kMxBM * kMxRowB, sf = b + NT * kMxRowB;
          const uint32_t sft = tmem + C::kSfCol + (it & 1) * 16;
          const int steps = min(4, (nb + 1) / 2 - 4 * k);
          for (int h = 0; h < (steps + 1) / 2; ++h) {
            ptx::tmem_cp_32x128(sft + 4 * h, ptx::rows16_desc(sf + 512 * h));
            ptx::tmem_cp_32x128(sft + 8 + 4 * h, ptx::rows16_desc(sf + kMxSfB + 512 * h));
          }
          const uint64_t da = ptx::sw128_desc(a, kHiK), db = ptx::sw128_desc(b, kHiK);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < steps)
              ptx::mma_mxf4_ss(d_tmem, da + 2 * q, db + 2 * q, ptx::idesc_mxf4(kMxBM, NT, 2 * (q & 1)),
                               sft + 4 * (q >> 1), sft + 8 + 4 * (q >> 1), k > 0 || q > 0);
          ptx::mma_commit(&bars->empty[s]);
        }
        if (ok) ptx::mma_commit(&bars->s_full[buf]);
      }
      if (!ok) mx_timeout(status, bars);
      if (*abort) {  // wait for the products already issued before TMEM is freed
        ptx::mma_commit(&bars->drain);
        ptx::mbar_drain(&bars->drain, 0);
      }
    }
  } else if (warp >= 4) {
    constexpr int kColsWarp = NT * 4 / C::kEpiWarps;          // columns a warp drains
    constexpr int kChunk32 = kColsWarp < 32 ? 16 : 32;
    const int q = warp & 3, c0 = ((warp - 4) >> 2) * kColsWarp;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    uint32_t j = 0;
    for (int64_t t = blockIdx.x; t < ntiles && !*abort; t += gridDim.x, ++j) {
      const int64_t nt = t / mtiles;
      const int64_t m0 = (t - nt * mtiles) * NT;
      const uint32_t buf = j & 1;
      const int64_t row = nt * kMxBM + q * 32 + lane;
      const float bv = bias && row < n ? __ldg(bias + row) : 0.f;
      if (!ptx::mbar_wait_warp(&bars->s_full[buf], (j >> 1) & 1, abort)) {
        mx_timeout(status, bars);
        break;
      }
      ptx::tc_fence_after();
#pragma unroll
      for (int c = 0; c < kColsWarp; c += kChunk32) {
        uint32_t u[kChunk32];
        if constexpr (kChunk32 == 32) ptx::tmem_ld32(tmem + lane_base + buf * NT + c0 + c, u);
        else ptx::tmem_ld16(tmem + lane_base + buf * NT + c0 + c, u);
        ptx::tmem_wait_ld();
        if (c + kChunk32 == kColsWarp) {  // all in registers: hand the accumulator back
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->s_empty[buf]);
        }
        const int64_t mc = m0 + c0 + c;
        T* p = out + mc * ldo + row;
        if (row < n) {
          if (mc + kChunk32 <= m) {
#pragma unroll
            for (int e = 0; e < kChunk32; ++e, p += ldo) mx_st(p, fmaf(alpha, __uint_as_float(u[e]), bv));
          } else {
#pragma unroll
            for (int e = 0; e < kChunk32; ++e, p += ldo)
              if (mc + e < m) mx_st(p, fmaf(alpha, __uint_as_float(u[e]), bv));
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kCols);
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn mx_encode_tiled() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                       cudaSuccess && q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
  }();
  return fn;
}

// Rows of codes as boxes of 128 bytes x `box_rows`; what lies beyond a row or the last row is 0.
bool mx_tmap(CUtensorMap* map, const uint8_t* codes, int nb, int64_t rows, int box_rows) {
  EncodeTiledFn enc = mx_encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)nb * 16, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)nb * 16};
  const cuuint32_t box[2] = {kMxRowB, (cuuint32_t)box_rows};
  const cuuint32_t one[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct MxArgs {
  const uint8_t *qc, *qs, *xc, *xs;
  int64_t m, n;
  int nb;
  float alpha;
  const float* bias;
  void* out;
  int64_t ldo;
  int* status;
  cudaStream_t s;
};

template <int NT, typename T>
cudaError_t mx_scores(const MxArgs& a) {
  using C = MxCfg<NT>;
  static_assert(C::kStages >= 4 && C::kStages <= 10 && C::kSfCol + 32 <= C::kCols, "tile");
  constexpr int smem = 1024 + C::kStages * C::kStage + (int)sizeof(MxBars);
  static_assert(smem <= 227 * 1024, "shared memory");
  CUtensorMap tmx, tmq;
  if (!mx_tmap(&tmx, a.xc, a.nb, a.n, kMxBM) || !mx_tmap(&tmq, a.qc, a.nb, a.m, NT))
    return cudaErrorInvalidValue;
  auto* k = mx4_scores_kernel<NT, T>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t mt = (a.m + NT - 1) / NT, tiles = (a.n + kMxBM - 1) / kMxBM * mt;
  k<<<(unsigned)(tiles < sms ? tiles : sms), C::kThreads, smem, a.s>>>(
      tmx, tmq, a.xs, a.qs, a.n, a.m, a.nb, tiles, (int)mt, a.alpha, a.bias, static_cast<T*>(a.out),
      a.ldo, a.status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t mx_scores_nt(const MxArgs& a) {
  if (a.m <= 16) return mx_scores<16, T>(a);
  if (a.m <= 32) return mx_scores<32, T>(a);
  if (a.m <= 64) return mx_scores<64, T>(a);
  return mx_scores<128, T>(a);
}

unsigned mx_grid(int64_t groups) {
  const int64_t blocks = (groups + kMxThreads / 32 - 1) / (kMxThreads / 32);
  return (unsigned)(blocks < (1 << 30) ? blocks : (1 << 30));
}

}  // namespace

// ------------------------------------------------------------------ launchers
cudaError_t launch_mx4_encode(const void* X, int x_dtype, int64_t n, int D, int64_t ldx,
                              uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  const int nb = (D + 31) / 32, nkc = (nb + 3) / 4;
  const int64_t groups = (n + 127) / 128 * 32 * nkc;
  const unsigned grid = mx_grid(groups);
  const size_t eb = x_dtype == FGMM_F32 ? 4 : 2;
  const bool vec = (uintptr_t)X % (4 * eb) == 0 && ldx % 4 == 0;
  if (x_dtype == FGMM_F32) {
    auto* k = vec ? mx4_encode_kernel<float, true> : mx4_encode_kernel<float, false>;
    k<<<grid, kMxThreads, 0, s>>>(static_cast<const float*>(X), n, D, ldx, nb, nkc, groups, codes,
                                  scales);
  } else {
    auto* k = vec ? mx4_encode_kernel<__nv_bfloat16, true> : mx4_encode_kernel<__nv_bfloat16, false>;
    k<<<grid, kMxThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(X), n, D, ldx, nb, nkc, groups,
                                  codes, scales);
  }
  return cudaGetLastError();
}

cudaError_t launch_mx4_decode(const uint8_t* codes, const uint8_t* scales, int64_t n, int D,
                              void* out, int out_dtype, int64_t ldo, cudaStream_t s) {
  const int nb = (D + 31) / 32, nkc = (nb + 3) / 4;
  const int64_t groups = (n + 127) / 128 * 32 * nkc;
  const unsigned grid = mx_grid(groups);
  const size_t eb = out_dtype == FGMM_F32 ? 4 : 2;
  const bool vec = (uintptr_t)out % (4 * eb) == 0 && ldo % 4 == 0;
  if (out_dtype == FGMM_F32) {
    auto* k = vec ? mx4_decode_kernel<float, true> : mx4_decode_kernel<float, false>;
    k<<<grid, kMxThreads, 0, s>>>(codes, scales, n, D, nb, nkc, groups, static_cast<float*>(out),
                                  ldo);
  } else {
    auto* k = vec ? mx4_decode_kernel<__nv_bfloat16, true> : mx4_decode_kernel<__nv_bfloat16, false>;
    k<<<grid, kMxThreads, 0, s>>>(codes, scales, n, D, nb, nkc, groups,
                                  static_cast<__nv_bfloat16*>(out), ldo);
  }
  return cudaGetLastError();
}

cudaError_t launch_mx4_scores(const uint8_t* q_codes, const uint8_t* q_scales, int64_t m,
                              const uint8_t* codes, const uint8_t* scales, int64_t n, int D,
                              float alpha, const float* bias, void* out, int out_dtype,
                              int64_t ldo, int* status, cudaStream_t s) {
  const MxArgs a = {q_codes, q_scales, codes, scales, m, n, (D + 31) / 32, alpha, bias, out, ldo,
                    status, s};
  return out_dtype == FGMM_F32 ? mx_scores_nt<float>(a) : mx_scores_nt<__nv_bfloat16>(a);
}

}  // namespace fgmm
