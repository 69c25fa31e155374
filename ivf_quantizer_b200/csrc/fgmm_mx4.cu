// 4-bit codes of vectors (OCP Microscaling Formats v1.0, MXFP4: blocks of 32 e2m1 codes with
// one e8m0 scale) and the scores of queries against them.  The layout of codes and scales is
// that of include/fgmm.h.
//
//   encode  reads 4 (or 2) bytes a value, writes 17/32: bound by reading
//   decode  the reverse: bound by writing
//   scores  out = alpha Q X^T + bias over the decoded values
#include <cuda_bf16.h>

#include "fgmm_internal.h"

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

// Scores on CUDA cores: a 64 x 64 tile of outputs a CTA, one block of 32 dimensions at a time
// decoded into shared memory, 4 x 4 outputs a thread.
template <typename T>
__global__ void __launch_bounds__(256)
    mx4_scores_simt_kernel(const uint8_t* __restrict__ qc, const uint8_t* __restrict__ qs, int64_t m,
                           const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                           int64_t n, int nb, float alpha, const float* __restrict__ bias,
                           T* __restrict__ out, int64_t ldo, int64_t ntiles_n) {
  __shared__ float sq[32][68], sx[32][68];
  const int nkc = (nb + 3) / 4;
  const int64_t m0 = (int64_t)(blockIdx.x / ntiles_n) * 64, n0 = (blockIdx.x % ntiles_n) * 64;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float acc[4][4] = {};
  for (int b = 0; b < nb; ++b) {
    // thread: 8 codes of one row of each side
    const int r = tid >> 2, part = tid & 3;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int64_t row = (side ? n0 : m0) + r;
      const uint8_t* codes = side ? xc : qc;
      const uint8_t* scales = side ? xs : qs;
      float v[8] = {};
      if (row < (side ? n : m)) {
        const float s = mx_scale(scales[((row >> 7) * nkc + (b >> 2)) * 512 + (row & 31) * 16 +
                                        ((row & 127) >> 5) * 4 + (b & 3)]);
        const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + row * ((int64_t)nb * 16) +
                                                              b * 16 + part * 4);
        float lo[4], hi[4];
        mx_values4(c, lo);
        mx_values4(c >> 16, hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = lo[j] * s, v[4 + j] = hi[j] * s;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) (side ? sx : sq)[part * 8 + j][r] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      float a[4], c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = sq[k][ty * 4 + j], c[j] = sx[k][tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], c[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = m0 + ty * 4 + i, col = n0 + tx + 16 * j;
      if (row < m && col < n)
        mx_st(out + row * ldo + col, fmaf(alpha, acc[i][j], bias ? bias[col] : 0.f));
    }
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
  (void)status;
  const int nb = (D + 31) / 32;
  const int64_t tn = (n + 63) / 64, tiles = tn * ((m + 63) / 64);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  if (out_dtype == FGMM_F32)
    mx4_scores_simt_kernel<float><<<(unsigned)tiles, 256, 0, s>>>(
        q_codes, q_scales, m, codes, scales, n, nb, alpha, bias, static_cast<float*>(out), ldo, tn);
  else
    mx4_scores_simt_kernel<__nv_bfloat16><<<(unsigned)tiles, 256, 0, s>>>(
        q_codes, q_scales, m, codes, scales, n, nb, alpha, bias, static_cast<__nv_bfloat16*>(out),
        ldo, tn);
  return cudaGetLastError();
}

}  // namespace fgmm
