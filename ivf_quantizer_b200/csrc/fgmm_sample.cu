// One draw per row of scores from its truncated softmax (temperature, top-k, top-p, min-p) with
// given uniforms.  The definition is that of fgmm_sample_logits in include/fgmm.h.
//
// Weights are 64-bit integers, w_i = round(2^40 exp((l_i - max l) / T)), so every sum is exact and
// independent of its order: the draw is reproducible, and ties of equal logits are exact.
// 2^40 leaves 2^22 tokens room in 63 bits; the error of a sum of n weights is at most n / 2 units.
//
// The tokens that top-k, top-p and min-p keep are a prefix of the order (logit descending, index
// ascending).  Tokens are numbered by that order with a 64-bit place (inverted key of the logit in
// the upper half, index in the lower half), and a truncation is the place of the last kept token.
// It is found by a histogram over log2 weights (bins of 1/32 down to weight 2^-41); the tokens of
// the bin that holds the border are sorted.  A bin too full for that is split by histograms over
// places first.
//
// A cluster of C CTAs takes a row, a contiguous slice each.  Steps, each ending in an exchange over
// the cluster:
//   maximum | [histogram, border]  for top-k, then for top-p | kept weight of every warp's
//   contiguous part | the warp whose part holds the target finds the token by a scan.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include "fgmm_internal.h"

namespace fgmm {
namespace {

namespace cg = cooperative_groups;

constexpr double kSmOne = 1099511627776.0;  // 2^40
constexpr uint64_t kSmAll = ~0ull;          // border that keeps everything

// The values of 16 bytes of a row, in groups of four.
template <typename T>
struct SmVec;
template <>
struct SmVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& t, int, float (&v)[4]) {
    v[0] = __uint_as_float(t.x), v[1] = __uint_as_float(t.y);
    v[2] = __uint_as_float(t.z), v[3] = __uint_as_float(t.w);
  }
  static __device__ __forceinline__ void put(uint32_t (&w)[4], int j, float x) {
    w[j] = __float_as_uint(x);
  }
  static constexpr uint32_t kMinusInf = 0xff800000u;
};
template <>
struct SmVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& t, int g, float (&v)[4]) {
    const uint32_t a = g ? t.z : t.x, b = g ? t.w : t.y;
    v[0] = __uint_as_float(a << 16), v[1] = __uint_as_float(a & 0xffff0000u);
    v[2] = __uint_as_float(b << 16), v[3] = __uint_as_float(b & 0xffff0000u);
  }
  static __device__ __forceinline__ void put(uint32_t (&w)[4], int j, __nv_bfloat16 x) {
    const uint32_t b = __bfloat16_as_ushort(x), at = 16 * (j & 1);
    w[j >> 1] = (w[j >> 1] & ~(0xffffu << at)) | b << at;
  }
  static constexpr uint32_t kMinusInf = 0xff80ff80u;
};

// Order-preserving integer of a logit; -0 and +0 are one value.
__device__ __forceinline__ uint32_t sm_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float sm_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ uint64_t sm_place(float x, uint32_t i) {
  return (uint64_t)(~sm_key(x)) << 32 | i;
}
__device__ __forceinline__ float sm_place_value(uint64_t c) { return sm_value(~(uint32_t)(c >> 32)); }

__device__ __forceinline__ float sm_max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// (double)x with infinity read as the largest finite value, so that a row whose maximum is infinite
// needs no case of its own (only its infinite logits are not below `least`).
__device__ __forceinline__ double sm_double(float x) { return (double)fminf(x, 3.402823466e38f); }

// What a row's weights need.
struct SmRow {
  float top, least;                         // logits below least weigh nothing (below 2^-41)
  double topd, c;                           // c = 32 log2(e) / T
};

// 2^(40 + j / 32)
__device__ const double kSmTable[32] = {
    1099511627776.0, 1123587797336.3408, 1148191166360.5662, 1173333279013.7073,
    1199025932245.0925, 1225281181323.604, 1252111345494.1387, 1279529013757.9299,
    1307547050779.4426, 1336178602922.6121, 1365437104419.2583, 1395336283672.5735,
    1425890169698.6345, 1457113098708.9692, 1489019720837.26, 1521625007013.345,
    1554944255987.7375, 1588993101509.9658, 1623787519664.0955, 1659343836364.8796,
    1695678735018.0535, 1732809264348.3684, 1770752846399.0352, 1809527284706.3352,
    1849150772653.2297, 1889641902005.8923, 1931019671637.1631, 1973303496441.0256,
    2016513216442.283, 2060669106105.7107, 2105791883849.0532, 2151902721764.3281};

constexpr double kSmMagic = 6755399441055744.0;  // 1.5 2^52: a sum's low word is the rounded integer
constexpr float kSmColdest = 8.271806125530277e-25f;  // 2^-80: logits that differ by 2^-74 or more differ
                                            // in weight by more than 2^-42 at any lower temperature too
constexpr int kSmBins = 1344;               // 32 bins a factor of two, down to 2^-41.3 and 2^-42

// -32 log2 of the weight of a logit above the floor, rounded: its bin.
__device__ __forceinline__ int sm_bin(float x, const SmRow& r) {
  return -__double2loint(fma(sm_double(x) - r.topd, r.c, kSmMagic));
}
// 2^40 2^(y / 32), y = (x - top) c in [-1322, 0], and the bin -round(y).  y = n + f with |f| <= 1/2;
// 2^(f / 32) by its Taylor series to f^5 (remainder 2^-48); table[j] = 2^(40 + j / 32), whose exponent
// takes n / 32.  The result is p t, before its rounding.
__device__ __forceinline__ void sm_exp(float x, const SmRow& r, const double* table, int& bin,
                                       double& p, double& t) {
  const double d = sm_double(x) - r.topd;
  const double k = fma(d, r.c, kSmMagic);
  const double f = fma(d, r.c, kSmMagic - k);
  p = 3.97370998454941609e-11;       // (ln 2 / 32)^5 / 5!
  p = fma(p, f, 9.17256270182464302e-09);
  p = fma(p, f, 1.69385097243718210e-06);
  p = fma(p, f, 2.34596198202246799e-04);
  p = fma(p, f, 2.16608493924982902e-02);
  p = fma(p, f, 1.0);
  const int n = __double2loint(k);
  t = table[n & 31];
  t = __hiloint2double(__double2hiint(t) + (n >> 5) * (1 << 20), __double2loint(t));
  bin = -n;
}
// The weight of a logit, and its bin.
__device__ __forceinline__ uint64_t sm_weight(float x, const SmRow& r, const double* table, int& bin) {
  double p, t;
  sm_exp(x, r, table, bin, p, t);
  const double m = fma(p, t, 4503599627370496.0);   // 2^52: the mantissa holds the rounded product
  return (uint64_t)__double_as_longlong(m) & 0xfffffffffffffull;
}

// min-p: the least weight it keeps, and a logit that is surely below every logit of that weight, so
// that the comparison of weights decides alone.
__device__ __forceinline__ uint64_t sm_min_weight(float mp) {
  return (uint64_t)__double2ull_ru((double)mp * kSmOne);
}
__device__ __forceinline__ float sm_min_logit(uint64_t least, float t, const SmRow& r) {
  if (least <= 1) return r.least;           // every weight that is not 0
  // what rounds to `least` is least - 1/2 and more; the slack, 1e-5 and 2e-5 of the logarithm (at most 28),
  // covers the rounding of the argument (6e-8), two ulps of __log2f (2^-22 near 1, 5e-6 at 41) and the products'
  const float down = fmaf(__log2f((float)(((double)least - 0.5) / kSmOne)), 0.6931482f * 1.00001f, -1e-5f) * t;
  return __double2float_rd((double)r.top + (double)down * 1.00001 - 1e-5 * (double)t);
}
// Bounds of a row's parameters (NaN fails them).
__device__ __forceinline__ bool sm_valid(float t, float p, float mp, double u) {
  return t >= 0.f && t < CUDART_INF_F && p > 0.f && p <= 1.f && mp >= 0.f && mp <= 1.f && u >= 0.0 &&
         u < 1.0;
}
__device__ __forceinline__ SmRow sm_row(float top, float t) {
  SmRow r;
  r.top = top;
  r.topd = sm_double(top);
  r.c = t > 0.f ? 46.166241308446828 / (double)t : 0.0;
  r.least = fminf(__double2float_ru((double)top - 28.62 * (double)t), top);
  return r;
}
__device__ __forceinline__ float sm_prob(float x, const SmRow& r, const double* table, float t,
                                         uint64_t total) {
  if (t == 0.f) return 1.f;
  int bin;
  double p, e;
  sm_exp(x, r, table, bin, p, e);
  return (float)(p * e / (double)total);
}

constexpr int kSmList = kSmBins * 12 / 8;    // tokens of a border bin that are ranked: what a histogram's room holds

template <int THREADS>
struct SmShared {
  static constexpr int kWarps = THREADS / 32;
  uint4 ends[2];
  // this CTA's histogram (mass in two words, number); then, in CTA 0, the list that is sorted
  union {
    struct { uint32_t lo[kSmBins], hi[kSmBins], cnt[kSmBins]; } h;
    uint64_t list[kSmList];
  };
  uint64_t m0[kSmBins];                     // the cluster's
  uint32_t c0[kSmBins];
  double table[32];
  uint64_t wsum[kWarps], wmass[kWarps];
  uint32_t wcnt[kWarps];
  float wmax[kWarps];
  float part_max[8];
  uint64_t part_lo, part_hi;
  uint64_t few[32], sums[8 * kWarps];
  uint64_t above_mass, out_place;
  uint32_t above_cnt, bin_cnt, nlist, nfew;
  int bin;
  uint64_t total, before;
  int owner;
};

struct SmArgs {
  const void* logits;
  int V;
  int64_t ld;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
  const double* u;
  int32_t* ids;
  float* prob;
  int slice;                                // values a CTA takes
};

template <typename T, int THREADS, bool RES>
struct Sampler {
  using S = SmShared<THREADS>;
  using V = SmVec<T>;
  static constexpr int W = THREADS / 32;
  static constexpr int kList = sizeof(S::list) / 8;
  S& s;
  cg::cluster_group cluster;
  int C, rank;
  const T* src;                             // the slice
  const uint4* data;                        // its 16-byte vectors: in shared memory, or in place
  int first, len, phase;                    // slice: first index, length, unused leading values
  int nvec, vpw;                            // vectors of the slice, vectors a warp
  int lane, warp;
  SmRow r;

  __device__ __forceinline__ void sync() {
    if (C == 1) __syncthreads();
    else cluster.sync();
  }
  template <typename U>
  __device__ __forceinline__ U* at(U* p, int q) {
    return C == 1 ? p : cluster.map_shared_rank(p, q);
  }

  // The first and the last vector of the slice hold values outside it, which read as -inf: they
  // are put together once (one thread each).
  __device__ __forceinline__ void make_ends() {
    if (threadIdx.x < 2 && nvec > 0) {
      const int v = threadIdx.x ? nvec - 1 : 0;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = V::kMinusInf;
#pragma unroll
      for (int j = 0; j < V::N; ++j) {
        const int i = v * V::N + j - phase;
        if (i >= 0 && i < len) V::put(w, j, src[i]);
      }
      s.ends[threadIdx.x] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
  }
  // Vector v of the slice from memory.
  __device__ __forceinline__ uint4 fetch(const uint4* g, int v) const {
    const bool inner = (unsigned)(v - 1) < (unsigned)(nvec - 2);
    const uint4* p = inner ? g + v : &s.ends[v > 0];
    return *p;
  }
  __device__ __forceinline__ uint4 raw(int v) const { return RES ? data[v] : fetch(data, v); }
  // Index of the first value of group g of vector v.
  __device__ __forceinline__ uint32_t index(int v, int g) const {
    return (uint32_t)(first + v * V::N + 4 * g - phase);
  }
  // f(four values, index of the first) for the groups of the slice that hold a value in [from, to]
  // (WINDOW) or of at least `from`, each warp its own contiguous part.
  template <bool WINDOW = false, typename F>
  __device__ __forceinline__ void each(float from, F f, float to = 0.f) {
    constexpr int U = RES ? 1 : 4;          // loads in flight
    const int v1 = min(nvec, (warp + 1) * vpw);
    for (int v = warp * vpw + lane; v < v1; v += 32 * U) {
      uint4 q[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        q[i] = raw(min(v + 32 * i, v1 - 1));
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int g = 0; g < V::N / 4; ++g) {
          float x[4];
          V::get(q[i], g, x);
          bool hit;
          if constexpr (WINDOW) {
            hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) hit |= x[e] >= from && x[e] <= to;
          } else {
            hit = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= from;
          }
          if (hit && (i == 0 || v + 32 * i < v1)) f(x, index(v + 32 * i, g));
        }
    }
  }
  // The weights of four logits (of which those that count are in [least, top]) and their bins.
  __device__ __forceinline__ void weights(const float (&x)[4], uint64_t (&w)[4], int (&bin)[4]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = sm_weight(x[j], r, s.table, bin[j]);
  }

  __device__ __forceinline__ void clear() {
    for (int b = threadIdx.x; b < kSmBins; b += THREADS) s.h.lo[b] = s.h.hi[b] = s.h.cnt[b] = 0u;
    __syncthreads();
  }
  // lo, hi: the two words of a 64-bit sum
  static __device__ __forceinline__ void add(uint32_t* lo, uint32_t* hi, uint64_t w) {
    const uint32_t l = (uint32_t)w, old = atomicAdd(lo, l);
    const uint32_t h = (uint32_t)(w >> 32) + (old + l < old ? 1u : 0u);
    if (h) atomicAdd(hi, h);
  }
  // The cluster's histogram in every CTA.
  __device__ void exchange(bool mass, bool count) {
    sync();
    if (threadIdx.x == 0) s.nlist = s.nfew = 0u;
    if (C == 1) {
      for (int b = threadIdx.x; b < kSmBins; b += THREADS) {
        s.m0[b] = ((uint64_t)s.h.hi[b] << 32) + s.h.lo[b];
        s.c0[b] = s.h.cnt[b];
      }
      __syncthreads();
      return;
    }
    const int seg = kSmBins / C;
    for (int i = threadIdx.x; i < seg; i += THREADS) {
      const int b = rank * seg + i;
      uint32_t lo[8], hi[8], n[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {         // all reads in flight together
        lo[q] = q < C && mass ? *at(&s.h.lo[b], q) : 0u;
        hi[q] = q < C && mass ? *at(&s.h.hi[b], q) : 0u;
        n[q] = q < C && count ? *at(&s.h.cnt[b], q) : 0u;
      }
      uint64_t m = 0;
      uint32_t c = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) m += ((uint64_t)hi[q] << 32) + lo[q], c += n[q];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < C) *at(&s.m0[b], q) = m, *at(&s.c0[b], q) = c;
    }
    sync();
  }
  // First bin at which the running number reaches k, or the running mass reaches need (s.bin,
  // kSmBins if none does), what is before it and how many tokens it holds.
  __device__ void pick(bool by_count, uint32_t k, double need, uint64_t above_mass, uint32_t above_cnt) {
    constexpr int PER = (kSmBins + THREADS - 1) / THREADS;
    const int b0 = threadIdx.x * PER, b1 = min(b0 + PER, kSmBins);
    uint64_t msum = 0;
    uint32_t csum = 0;
    for (int b = b0; b < b1; ++b) msum += s.m0[b], csum += s.c0[b];
    uint64_t mi = msum;
    uint32_t ci = csum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t a = __shfl_up_sync(0xffffffffu, mi, o);
      const uint32_t b = __shfl_up_sync(0xffffffffu, ci, o);
      if (lane >= o) mi += a, ci += b;
    }
    const uint64_t mw = __shfl_sync(0xffffffffu, mi, 31);
    const uint32_t cw = __shfl_sync(0xffffffffu, ci, 31);
    if (lane == 0) s.wmass[warp] = mw, s.wcnt[warp] = cw;
    if (threadIdx.x == 0) s.bin = kSmBins;
    __syncthreads();
    uint64_t before = lane < warp ? s.wmass[lane] : 0ull;      // (W <= 32)
    uint32_t cbefore = lane < warp ? s.wcnt[lane] : 0u;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, o);
      cbefore += __shfl_xor_sync(0xffffffffu, cbefore, o);
    }
    mi += __shfl_sync(0xffffffffu, before, 0), ci += __shfl_sync(0xffffffffu, cbefore, 0);
    uint64_t run_m = above_mass + mi - msum;
    uint32_t run_c = above_cnt + ci - csum;
    for (int b = b0; b < b1; ++b) {
      const bool was = by_count ? run_c >= k : (double)run_m >= need;
      const uint64_t nm = run_m + s.m0[b];
      const uint32_t nc = run_c + s.c0[b];
      if (!was && (by_count ? nc >= k : (double)nm >= need)) {
        s.bin = b;
        s.bin_cnt = nc - run_c;
        s.above_mass = run_m;
        s.above_cnt = run_c;
      }
      run_m = nm, run_c = nc;
    }
    __syncthreads();
  }

  // CTA 0: among the n places of the list, the one at which the running number reaches k, or the
  // running mass reaches need, in ascending order; tells every CTA.  Histograms over places (in
  // m0, c0) narrow the list down to at most 32 of them, which one warp ranks.
  __device__ void resolve(uint32_t n, bool by_count, uint32_t k, double need, uint64_t above,
                          uint32_t above_cnt) {
    const uint32_t all = n;
    uint64_t lo = 0, hi = kSmAll;
    if (n > 32) {
      lo = kSmAll, hi = 0;
      for (uint32_t i = threadIdx.x; i < all; i += THREADS) lo = min(lo, s.list[i]), hi = max(hi, s.list[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, (uint64_t)__shfl_xor_sync(0xffffffffu, lo, o));
        hi = max(hi, (uint64_t)__shfl_xor_sync(0xffffffffu, hi, o));
      }
      if (lane == 0) s.wsum[warp] = lo, s.wmass[warp] = hi;
      __syncthreads();
      lo = s.wsum[lane % W], hi = s.wmass[lane % W];
#pragma unroll
      for (int o = 1; o < W; o <<= 1) {
        lo = min(lo, (uint64_t)__shfl_xor_sync(0xffffffffu, lo, o));
        hi = max(hi, (uint64_t)__shfl_xor_sync(0xffffffffu, hi, o));
      }
    }
    while (n > 32) {
      const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 10);   // at most 1024 parts
      for (int b = threadIdx.x; b < kSmBins; b += THREADS) s.m0[b] = 0ull, s.c0[b] = 0u;
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < all; i += THREADS) {
        const uint64_t c = s.list[i];
        if (c >= lo && c <= hi) {
          const int b = (int)((c - lo) >> shift);
          int bin;
          atomicAdd(&s.c0[b], 1u);
          uint32_t* m = reinterpret_cast<uint32_t*>(&s.m0[b]);
          if (!by_count) add(m, m + 1, sm_weight(sm_place_value(c), r, s.table, bin));
        }
      }
      __syncthreads();
      pick(by_count, k, need, above, above_cnt);
      n = s.bin_cnt, above = s.above_mass, above_cnt = s.above_cnt;
      lo += (uint64_t)s.bin << shift;
      hi = lo + min(hi - lo, (uint64_t)((1ull << shift) - 1));
      __syncthreads();
    }
    for (uint32_t i = threadIdx.x; i < all; i += THREADS) {
      const uint64_t c = s.list[i];
      if (c >= lo && c <= hi) s.few[atomicAdd(&s.nfew, 1u)] = c;
    }
    __syncthreads();
    if (warp == 0) {
      const uint64_t mine = lane < (int)n ? s.few[lane] : kSmAll;
      int bin;
      const uint64_t w = by_count || lane >= (int)n ? 0ull : sm_weight(sm_place_value(mine), r, s.table, bin);
      uint64_t before = above;
      uint32_t rank_of = above_cnt;
      for (int j = 0; j < (int)n; ++j) {
        const uint64_t c = __shfl_sync(0xffffffffu, mine, j), v = __shfl_sync(0xffffffffu, w, j);
        if (c < mine) before += v, ++rank_of;
      }
      const bool is = by_count ? rank_of + 1 == k : (double)before < need && (double)(before + w) >= need;
      if (is && lane < (int)n)
        for (int q = 0; q < C; ++q) *at(&s.out_place, q) = mine;
    }
  }

  // The logits of a bin, a few roundings wider: which of them are in it is asked one by one.
  __device__ __forceinline__ void window(int bin, float from, float& low, float& high) const {
    const double unit = 1.0 / r.c, x0 = r.topd + (-bin - 0.5) * unit, x1 = x0 + unit;
    const double slack = 1e-6 * (fabs(r.topd) + fabs(x0) + unit);
    low = fmaxf(from, __double2float_rd(x0 - slack)), high = __double2float_ru(x1 + slack);
  }

  // Block-wide sum, every thread receives it.
  __device__ __forceinline__ uint64_t sum_all(uint64_t w) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    __syncthreads();
    if (lane == 0) s.wsum[warp] = w;
    __syncthreads();
    w = s.wsum[lane % W];
#pragma unroll
    for (int o = 1; o < W; o <<= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    return w;
  }

  // The whole rest of a row whose border lies in bin `bin`, when so few tokens (n <= THREADS)
  // lie in the bins down to it that a thread can take one: CTA 0 collects them, and every thread
  // counts the others against its own, first by place (top-k, top-p), then by index (the draw).
  // `whole`: the mass that top-p refers to, 0 for that of the k tokens.
  __device__ void few(int bin, uint32_t n, uint32_t k, uint64_t whole, float p, uint64_t least, double u,
                      float from, const SmArgs& a, int64_t rw, float t);

  // The place of the last token that a truncation keeps: the k-th (by_count), or that at which the
  // running mass reaches need.  The border's bin has been picked from the cluster's histogram; `from`:
  // tokens below are not in it.
  __device__ uint64_t find(bool by_count, uint32_t k, double need, float from, uint64_t limit) {
    if (s.bin == kSmBins) return limit;     // all that weighs anything is kept
    const int bin0 = s.bin;
    uint64_t above = s.above_mass;
    uint32_t above_cnt = s.above_cnt;
    float low, high;
    window(bin0, from, low, high);
    uint64_t lo = 0, hi = kSmAll;
    for (int level = 0;; ++level) {
      auto member = [&](float x, uint32_t i, uint64_t& c) {
        if (x > high || sm_bin(x, r) != bin0) return false;
        c = sm_place(x, i);
        return c >= lo && c <= hi && c <= limit;
      };
      // collect them in CTA 0 (the counters are 0 since the exchange); if they are too many for its
      // list, split them first
      each<true>(low, [&](const float (&x)[4], uint32_t i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint64_t c;
          if (x[e] >= low && member(x[e], i + e, c)) {
            const uint32_t j = atomicAdd(at(&s.nlist, 0), 1u);
            if (j < (uint32_t)kList) *at(&s.list[j], 0) = c;
          }
        }
      }, high);
      sync();
      const uint32_t n = *at(&s.nlist, 0);
      if (n <= (uint32_t)kList) {
        if (rank == 0) resolve(n, by_count, k, need, above, above_cnt);
        sync();
        return s.out_place;
      }
      if (level == 0) {                     // the range of places in the bin
        uint64_t a = kSmAll, b = 0;
        each<true>(low, [&](const float (&x)[4], uint32_t i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint64_t c;
            if (x[e] >= low && member(x[e], i + e, c)) a = min(a, c), b = max(b, c);
          }
        }, high);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          a = min(a, (uint64_t)__shfl_xor_sync(0xffffffffu, a, o));
          b = max(b, (uint64_t)__shfl_xor_sync(0xffffffffu, b, o));
        }
        if (lane == 0) s.wsum[warp] = a, s.wmass[warp] = b;
        __syncthreads();
        if (threadIdx.x == 0) {
          for (int q = 0; q < W; ++q) a = min(a, s.wsum[q]), b = max(b, s.wmass[q]);
          s.part_lo = a, s.part_hi = b;
        }
        sync();
        lo = kSmAll, hi = 0;
        for (int q = 0; q < C; ++q) lo = min(lo, *at(&s.part_lo, q)), hi = max(hi, *at(&s.part_hi, q));
      }
      const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 10);   // at most 1024 parts
      clear();
      each<true>(low, [&](const float (&x)[4], uint32_t i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint64_t c;
          if (x[e] >= low && member(x[e], i + e, c)) {
            const int b = (int)((c - lo) >> shift);
            int bin;
            if (by_count) atomicAdd(&s.h.cnt[b], 1u);
            else add(&s.h.lo[b], &s.h.hi[b], sm_weight(x[e], r, s.table, bin));
          }
        }
      }, high);
      exchange(!by_count, by_count);
      pick(by_count, k, need, above, above_cnt);
      const int bin = s.bin;
      above = s.above_mass, above_cnt = s.above_cnt;
      lo += (uint64_t)bin << shift;
      hi = lo + min(hi - lo, (uint64_t)((1ull << shift) - 1));
      __syncthreads();
    }
  }
};

template <typename T, int THREADS, bool RES>
__device__ void Sampler<T, THREADS, RES>::few(int bin, uint32_t n, uint32_t k, uint64_t whole, float p,
                                              uint64_t least, double u, float from, const SmArgs& a,
                                              int64_t rw, float t) {
  float low, high;
  window(bin, from, low, high);
  each(low, [&](const float (&x)[4], uint32_t i) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (x[e] >= low && (x[e] > high || sm_bin(x[e], r) <= bin)) {
        const uint32_t j = atomicAdd(at(&s.nlist, 0), 1u);
        if (j < (uint32_t)THREADS) *at(&s.list[j], 0) = sm_place(x[e], i + e);
      }
  });
  sync();                                   // the last access to another CTA's memory is before this
  if (rank != 0) return;
  // G lanes a token, each comparing it with every G-th
  int G = 1;
  while (G < 32 && 2 * G * n <= (uint32_t)THREADS) G *= 2;
  const uint32_t me = threadIdx.x / G, part = threadIdx.x % G;
  const uint64_t mine = me < n ? s.list[me] : kSmAll;
  const float x = sm_place_value(mine);
  int b;
  const uint64_t w = me < n ? sm_weight(x, r, s.table, b) : 0ull;
  if (part == 0 && me < n) s.m0[me] = w;
  __syncthreads();
  uint32_t before = 0;
  uint64_t mass = 0;
#pragma unroll 4
  for (uint32_t j = part; j < n; j += G)
    if (s.list[j] < mine) ++before, mass += s.m0[j];
  for (int o = 1; o < G; o <<= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    mass += __shfl_xor_sync(0xffffffffu, mass, o);
  }
  const uint64_t wk = before < k ? w : 0ull;
  const uint64_t in_k = sum_all(part == 0 ? wk : 0ull);   // (its barriers also end the reading of m0)
  if (whole == 0) whole = in_k;
  const bool kept = wk > 0 && wk >= least && (before == 0 || p >= 1.f || (double)mass < (double)p * (double)whole);
  if (part == 0 && me < n) s.m0[me] = kept ? w : 0ull;
  const uint64_t total = sum_all(part == 0 && kept ? w : 0ull);
  const uint64_t target = min((uint64_t)(u * (double)total), total - 1);
  uint64_t run = 0;
#pragma unroll 4
  for (uint32_t j = part; j < n; j += G)
    if ((uint32_t)s.list[j] < (uint32_t)mine) run += s.m0[j];
  for (int o = 1; o < G; o <<= 1) run += __shfl_xor_sync(0xffffffffu, run, o);
  if (kept && part == 0 && run <= target && run + w > target) {
    a.ids[rw] = (int32_t)(uint32_t)mine;
    if (a.prob) a.prob[rw] = sm_prob(x, r, s.table, t, total);
  }
}

template <typename T, int THREADS, bool RES>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) sample_kernel(const SmArgs a) {
  using Sm = Sampler<T, THREADS, RES>;
  using Vv = SmVec<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  SmShared<THREADS>& s = *reinterpret_cast<SmShared<THREADS>*>(smem);
  constexpr size_t kData = (sizeof(SmShared<THREADS>) + 15) / 16 * 16;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t rw = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float t = a.temperature ? a.temperature[rw] : 1.f;
  const float p = a.top_p ? a.top_p[rw] : 1.f;
  const float mp = a.min_p ? a.min_p[rw] : 0.f;
  const double un = a.u[rw];
  const int k = a.top_k ? a.top_k[rw] : 0;
  const bool bad = !sm_valid(t, p, mp, un);
  if (bad) {
    if (rank == 0 && tid == 0) {
      a.ids[rw] = -1;
      if (a.prob) a.prob[rw] = CUDART_NAN_F;
    }
    return;
  }
  // no CTA writes to another's memory before that one runs: arrive now, wait before the first write
  if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (t > 0.f) t = fmaxf(t, kSmColdest);
  if (tid < 32) s.table[tid] = kSmTable[tid];
  const int first = min(rank * a.slice, a.V), len = min(a.slice, a.V - first);
  const T* src = static_cast<const T*>(a.logits) + rw * a.ld + first;
  const int phase = (int)((uintptr_t)src % 16 / sizeof(T));
  const uint4* g = reinterpret_cast<const uint4*>(src - phase);
  uint4* data = reinterpret_cast<uint4*>(smem + kData);
  const int nvec = len > 0 ? (phase + len + Vv::N - 1) / Vv::N : 0;
  Sm z = {s, cluster, C, rank, src, RES ? data : g, first, len, phase, nvec,
          (nvec + Sm::W - 1) / Sm::W, lane, warp, {}};

  z.make_ends();
  // the maximum (NaN when there is one); RES: the slice goes to shared memory
  float best = -CUDART_INF_F;
  for (int v0 = tid; v0 < nvec; v0 += THREADS * 8) {
    uint4 q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (v0 + i * THREADS < nvec) q[i] = z.fetch(g, v0 + i * THREADS);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int v = v0 + i * THREADS;
      if (v < nvec) {
#pragma unroll
        for (int g = 0; g < Vv::N / 4; ++g) {
          float x[4];
          Vv::get(q[i], g, x);
          best = sm_max_nan(best, sm_max_nan(sm_max_nan(x[0], x[1]), sm_max_nan(x[2], x[3])));
        }
        if (RES) data[v] = q[i];
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = sm_max_nan(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) s.wmax[warp] = best;
  if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    for (int q = 0; q < Sm::W; ++q) best = sm_max_nan(best, s.wmax[q]);
    for (int q = 0; q < C; ++q) *z.at(&s.part_max[rank], q) = best;
  }
  z.sync();
  float top = s.part_max[0];
  for (int q = 1; q < C; ++q) top = sm_max_nan(top, s.part_max[q]);
  if (isnan(top) || top == -CUDART_INF_F) {
    if (rank == 0 && tid == 0) {
      a.ids[rw] = -1;
      if (a.prob) a.prob[rw] = isnan(top) ? CUDART_NAN_F : 0.f;
    }
    return;
  }
  z.r = sm_row(top, t);
  const SmRow r = z.r;

  // the border: place of the last kept token
  uint64_t border = kSmAll;
  float from = r.least;                     // the border's logit, or the least that weighs anything
  if (t == 0.f) {
    from = top;
    border = sm_place(top, 0xffffffffu);
  } else {
    if (k > 0 && k < a.V) {
      z.clear();
      z.each(from, [&](const float (&x)[4], uint32_t) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x[e] >= from) atomicAdd(&s.h.cnt[sm_bin(x[e], r)], 1u);
      });
      z.exchange(false, true);
      z.pick(true, (uint32_t)k, 0.0, 0ull, 0u);
      const uint32_t n = s.above_cnt + s.bin_cnt;
      if (s.bin < kSmBins && n <= (uint32_t)THREADS) {
        z.few(s.bin, n, (uint32_t)k, 0ull, p, sm_min_weight(mp), un, from, a, rw, t);
        return;
      }
      border = z.find(true, (uint32_t)k, 0.0, from, border);
      if (border != kSmAll) from = fmaxf(from, sm_place_value(border));
    }
    if (p < 1.f) {
      z.clear();
      const uint32_t il = (uint32_t)border;
      // rows in shared memory are short: there it pays to count as well, for few()
      const bool count = RES && border == kSmAll;
      z.each(from, [&](const float (&x)[4], uint32_t i) {
        uint64_t w[4];
        int bin[4];
        z.weights(x, w, bin);
        if (border == kSmAll) {             // (the usual case, kept short: this pass is bound by issue)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (x[e] >= from) {
              z.add(&s.h.lo[bin[e]], &s.h.hi[bin[e]], w[e]);
              if (count) atomicAdd(&s.h.cnt[bin[e]], 1u);
            }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (x[e] > from || (x[e] == from && i + e <= il))
              z.add(&s.h.lo[bin[e]], &s.h.hi[bin[e]], w[e]);
        }
      });
      z.exchange(true, count);
      uint64_t whole = 0, m = 0;
      for (int b = tid; b < kSmBins; b += THREADS) m += s.m0[b];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      if (lane == 0) s.wsum[warp] = m;
      __syncthreads();
      for (int q = 0; q < Sm::W; ++q) whole += s.wsum[q];
      __syncthreads();
      z.pick(false, 0u, (double)p * (double)whole, 0ull, 0u);
      const uint32_t n = s.above_cnt + s.bin_cnt;
      if (count && n <= (uint32_t)THREADS) {
        z.few(s.bin, n, UINT32_MAX, whole, p, sm_min_weight(mp), un, from, a, rw, t);
        return;
      }
      border = z.find(false, 0u, (double)p * (double)whole, from, border);
      if (border != kSmAll) from = fmaxf(from, sm_place_value(border));
    }
    if (mp > 0.f) from = fmaxf(from, sm_min_logit(sm_min_weight(mp), t, r));
  }
  const uint64_t least = t > 0.f ? sm_min_weight(mp) : 0ull;   // weight that min-p asks for
  // tokens above `from` count, and those at it up to index ib
  const uint32_t ib = border == kSmAll || sm_place_value(border) < from ? 0xffffffffu : (uint32_t)border;
  auto kept = [&](const float (&x)[4], uint32_t i, uint64_t (&w)[4]) {
    int bin[4];
    if (t == 0.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = 1ull;
    } else {
      z.weights(x, w, bin);
    }
    bool tie = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = x[e] >= from ? w[e] : 0ull;
      tie |= x[e] == from;
    }
    if (tie) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (x[e] == from && i + e > ib) w[e] = 0ull;
    }
    if (least > 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (w[e] < least) w[e] = 0ull;
    }
  };
  uint64_t mass = 0;
  z.each(from, [&](const float (&x)[4], uint32_t i) {
    uint64_t w[4];
    kept(x, i, w);
    mass += (w[0] + w[1]) + (w[2] + w[3]);
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  if (lane < C) *z.at(&s.sums[rank * Sm::W + warp], lane) = mass;
  z.sync();                                 // the last access to another CTA's memory is before this
  // the warp whose part holds the target
  if (tid < 32) {
    constexpr int PER = Sm::W * 8 / 32;     // sums a lane, in order
    uint64_t w[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int q = lane * PER + i;
      w[i] = q < C * Sm::W ? s.sums[q] : 0ull;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += w[i];
    uint64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t b = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += b;
    }
    const uint64_t total = __shfl_sync(0xffffffffu, inc, 31);
    const uint64_t target = t == 0.f ? 0ull : min((uint64_t)(un * (double)total), total - 1);
    uint64_t start = inc - sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (start <= target && start + w[i] > target) {
        s.owner = lane * PER + i;
        s.before = target - start;          // weight to pass inside the part
        s.total = total;
      }
      start += w[i];
    }
  }
  __syncthreads();
  if (s.owner != rank * Sm::W + warp) return;
  const uint64_t target = s.before;
  uint64_t run = 0;
  const int v1 = min(nvec, (warp + 1) * z.vpw);
  for (int v0 = warp * z.vpw; v0 < v1; v0 += 32) {
    const int v = v0 + lane;
    constexpr int G = Vv::N / 4;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    uint64_t w[G][4], sum = 0;
    if (v < v1) q = z.raw(v);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float x[4];
      Vv::get(q, g, x);
      kept(x, z.index(v, g), w[g]);
      sum += v < v1 ? (w[g][0] + w[g][1]) + (w[g][2] + w[g][3]) : 0ull;
    }
    uint64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t b = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += b;
    }
    uint64_t at = run + inc - sum;
    if (at <= target && at + sum > target) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float x[4];
        Vv::get(q, g, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (at <= target && at + w[g][e] > target) {
            a.ids[rw] = (int32_t)(z.index(v, g) + e);
            if (a.prob) a.prob[rw] = sm_prob(x[e], r, s.table, t, s.total);
          }
          at += w[g][e];
        }
      }
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
    if (run > target) break;
  }
}

// One warp a row, for rows of at most kSmWarpV values without top-k and top-p: a CTA a row spends
// its time on barriers there.  The row lies in shared memory, and loops are short: with the row in
// registers and every loop unrolled, the warps waited for instructions.
//
// us, a CTA and a warp a row, fp32, no cut / with min-p: 16384 rows x 128 69 / 72 and 24 / 20, x 1024 87 / 84
// and 73 / 35, x 1500 126 / 118 and 125 / 59, x 2000 144 / 129 and 286 / 76; 4096 x 1024 25 / 24 and 22 / 11.
// With min-p a warp is faster beyond 1024 as well, without a cut it is not, and a single row of 1024 without a
// cut takes it 9.9 against 5.1 (one of 256 5.4 and 4.9, of 128 4.1 and 4.7): one lane weighs 32 tokens.
constexpr int kSmWarpV = 1024, kSmWarps = 4;

template <typename T>
__global__ void __launch_bounds__(32 * kSmWarps) sample_warp_kernel(const SmArgs a, int64_t rows) {
  using Vv = SmVec<T>;
  constexpr int G = Vv::N / 4, NV = kSmWarpV / Vv::N + 1;   // groups a vector, vectors a row
  __shared__ uint4 data[kSmWarps][NV];
  __shared__ uint16_t list[kSmWarps][kSmWarpV];
  __shared__ double table[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rw = (int64_t)blockIdx.x * kSmWarps + warp;
  if (threadIdx.x < 32) table[threadIdx.x] = kSmTable[threadIdx.x];
  __syncthreads();
  if (rw >= rows) return;
  float t = a.temperature ? a.temperature[rw] : 1.f;
  const float mp = a.min_p ? a.min_p[rw] : 0.f;
  const double un = a.u[rw];
  const T* src = static_cast<const T*>(a.logits) + rw * a.ld;
  const int phase = (int)((uintptr_t)src % 16 / sizeof(T)), nvec = (phase + a.V + Vv::N - 1) / Vv::N;
  const uint4* g = reinterpret_cast<const uint4*>(src - phase);
  uint4* row = data[warp];
#pragma unroll 4
  for (int v = lane; v < nvec; v += 32)
    if (v * Vv::N >= phase && (v + 1) * Vv::N <= phase + a.V) row[v] = __ldg(g + v);
  const int v0 = lane ? nvec - 1 : 0;       // the ragged ends of the row
  if (lane < 2 && !(v0 * Vv::N >= phase && (v0 + 1) * Vv::N <= phase + a.V)) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = Vv::kMinusInf;
#pragma unroll
    for (int j = 0; j < Vv::N; ++j) {
      const int e = v0 * Vv::N + j - phase;
      if (e >= 0 && e < a.V) Vv::put(w, j, src[e]);
    }
    row[v0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  float top = -CUDART_INF_F;
  for (int v = lane; v < nvec; v += 32) {
    const uint4 q = row[v];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float x[4];
      Vv::get(q, h, x);
      top = sm_max_nan(top, sm_max_nan(sm_max_nan(x[0], x[1]), sm_max_nan(x[2], x[3])));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = sm_max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool bad = !sm_valid(t, 1.f, mp, un) || isnan(top);
  if (bad || top == -CUDART_INF_F) {
    if (lane == 0) {
      a.ids[rw] = -1;
      if (a.prob) a.prob[rw] = bad ? CUDART_NAN_F : 0.f;
    }
    return;
  }
  if (t > 0.f) t = fmaxf(t, kSmColdest);
  const SmRow r = sm_row(top, t);
  float from = r.least;
  if (t == 0.f) from = top;
  else if (mp > 0.f) from = fmaxf(from, sm_min_logit(sm_min_weight(mp), t, r));
  const uint64_t least = t > 0.f ? sm_min_weight(mp) : 0ull;   // weight that min-p asks for
  // the tokens that may be kept, in index order: most rows keep few, and their weights are then
  // computed by full warps
  const T* val = reinterpret_cast<const T*>(row) + phase;
  uint16_t* kept = list[warp];
  int n = 0;
#pragma unroll 4
  for (int i0 = 0; i0 < a.V; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < a.V && (float)val[i] >= from;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (in) kept[n + __popc(m & ((1u << lane) - 1u))] = (uint16_t)i;
    n += __popc(m);
  }
  __syncwarp();
  auto weight = [&](int j) -> uint64_t {
    if (j >= n) return 0ull;
    int bin;
    const uint64_t w = t == 0.f ? 1ull : sm_weight((float)val[kept[j]], r, table, bin);
    return w >= least ? w : 0ull;
  };
  // a contiguous run of the list a lane; then the lane whose run holds the target, by the whole warp
  const int per = (n + 31) / 32;
  uint64_t sum = 0;
  for (int i = 0, at = per > 0 ? lane % per : 0; i < per; ++i) {   // (starts apart: no two lanes on a bank)
    sum += weight(lane * per + at);
    if (++at == per) at = 0;
  }
  uint64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t b = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += b;
  }
  const uint64_t total = __shfl_sync(0xffffffffu, inc, 31);
  const uint64_t target = t == 0.f ? 0ull : min((uint64_t)(un * (double)total), total - 1);
  const int owner = __ffs(__ballot_sync(0xffffffffu, inc > target)) - 1;
  const uint64_t before = __shfl_sync(0xffffffffu, inc - sum, owner);
  const int j = owner * per + lane;
  const uint64_t w = lane < per ? weight(j) : 0ull;
  inc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t b = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += b;
  }
  if (w > 0 && before + inc > target && before + inc - w <= target) {
    const int i = kept[j];
    a.ids[rw] = i;
    if (a.prob) a.prob[rw] = sm_prob((float)val[i], r, table, t, total);
  }
}

template <typename T, int THREADS, bool RES>
cudaError_t sm_launch(const SmArgs& a, int64_t rows, int C, size_t smem, cudaStream_t st) {
  auto* k = sample_kernel<T, THREADS, RES>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename T>
cudaError_t sm_choose(SmArgs a, int64_t rows, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // threads: a row of up to 4096 tokens; slices in shared memory, two CTAs a SM; slices in place, four
  // (more rows side by side cover one another's barriers: 173 us against 182, 256 x 131072)
  constexpr int kSmall = 128, kLarge = 512, kLong = 256;
  constexpr size_t kFixedSmall = (sizeof(SmShared<kSmall>) + 15) / 16 * 16;
  constexpr size_t kFixed = (sizeof(SmShared<kLarge>) + 15) / 16 * 16;
  constexpr size_t kFixedLong = (sizeof(SmShared<kLong>) + 15) / 16 * 16;
  constexpr size_t kHalf = 113 * 1024;      // two CTAs a SM
  const auto bytes = [&](int C) { return ((size_t)((a.V + C - 1) / C) * sizeof(T) + 31) / 16 * 16; };
  if (a.V <= kSmWarpV && !a.top_k && !a.top_p) {
    sample_warp_kernel<T><<<(unsigned)((rows + kSmWarps - 1) / kSmWarps), 32 * kSmWarps, 0, st>>>(a, rows);
    return cudaGetLastError();
  }
  if (a.V <= 4096) {
    a.slice = a.V;
    return sm_launch<T, kSmall, true>(a, rows, 1, kFixedSmall + bytes(1), st);
  }
  // CTAs a row: while the rows leave SMs idle, and until a slice has at most 32768 tokens.  us with slices of
  // at most 16384 / 32768 / 65536 / 131072, top-p: fp32 256 x 50021 117 / 73 / 87 / 87, 256 x 131072 274 / 162 /
  // 174 / 249, 300 x 70000 214 / 155 / 117 / 120, 256 x 262144 (eight CTAs at most) - / 316 / 323 / 352; bf16
  // 256 x 131072 257 / 200 / 175 / 194, 1024 x 50021 378 / 278 / 251 / 250.  Fastest in fp32 but for rows just
  // above a power of two of slices; half as many tokens' bytes in bf16 would bear 65536
  int C = 1;
  while (C < 8 && (a.V / C > 32768 || (rows * C < sms && a.V / C > 4096))) C *= 2;
  a.slice = (a.V + C - 1) / C;
  if (rows * C > INT32_MAX) return cudaErrorInvalidValue;
  if (kFixed + bytes(C) <= kHalf)
    return sm_launch<T, kLarge, true>(a, rows, C, kFixed + bytes(C), st);
  return sm_launch<T, kLong, false>(a, rows, C, kFixedLong, st);
}

}  // namespace

// ------------------------------------------------------------------ launcher
cudaError_t launch_sample_logits(const void* logits, int dtype, int64_t rows, int V, int64_t ld,
                                 const float* temperature, const int32_t* top_k,
                                 const float* top_p, const float* min_p, const double* u,
                                 int32_t* ids, float* prob, cudaStream_t s) {
  const SmArgs a = {logits, V, ld, temperature, top_k, top_p, min_p, u, ids, prob, 0};
  return dtype == FGMM_F32 ? sm_choose<float>(a, rows, s) : sm_choose<__nv_bfloat16>(a, rows, s);
}

}  // namespace fgmm
