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
// It is found by histograms: first over logits (bins of equal width down to weight 2^-41), then,
// inside the bin that holds the border, over places, until so few tokens are left that they can be
// ranked against one another.
//
// A cluster of C CTAs takes a row; each keeps its contiguous slice of the row in shared memory,
// so the row is read once from memory.  Steps, each ending in an exchange over the cluster:
//   maximum (while loading) | [histogram, border]  twice at most | kept weight of every warp's
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

__device__ __forceinline__ float sm_ld(const float* p) { return __ldg(p); }
__device__ __forceinline__ float sm_ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// The values of 16 bytes of a row.
template <typename T>
struct SmVec;
template <>
struct SmVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& t, float (&v)[4]) {
    v[0] = __uint_as_float(t.x), v[1] = __uint_as_float(t.y);
    v[2] = __uint_as_float(t.z), v[3] = __uint_as_float(t.w);
  }
  static constexpr uint32_t kMinusInf = 0xff800000u;
};
template <>
struct SmVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& t, float (&v)[8]) {
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
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

// What a row's weights and bins need.
struct SmRow {
  float top, half_top, bin_scale;
  double topd, c;                           // c = log2(e) / T
};

// round(2^40 2^y) for y = (x - top) c in [-42, 0], 2^40 for the maximum itself (infinite or not):
// y = n + f with |f| <= 1/2, the Taylor series of 2^f to f^11 (remainder 2^-47), the exponent
// n + 40 added to that of the sum, and the rounding done by adding 2^52.
__device__ __forceinline__ uint64_t sm_weight(float x, const SmRow& r) {
  const double y = ((double)x - r.topd) * r.c;
  const double k = y + 6755399441055744.0;  // 1.5 2^52: the low word holds round(y)
  const double f = y - (k - 6755399441055744.0);
  double p = 4.4455382718708116e-10;        // ln(2)^11 / 11!
  p = fma(p, f, 7.0549116208011234e-09);
  p = fma(p, f, 1.0178086009239700e-07);
  p = fma(p, f, 1.3215486790144310e-06);
  p = fma(p, f, 1.5252733804059841e-05);
  p = fma(p, f, 1.5403530393381609e-04);
  p = fma(p, f, 1.3333558146428443e-03);
  p = fma(p, f, 9.6181291076284769e-03);
  p = fma(p, f, 5.5504108664821583e-02);
  p = fma(p, f, 2.4022650695910072e-01);
  p = fma(p, f, 6.9314718055994529e-01);
  p = fma(p, f, 1.0);
  const int n = __double2loint(k) + 40;
  const double w = __hiloint2double(__double2hiint(p) + (n << 20), __double2loint(p));
  const double m = w + 4503599627370496.0;  // 2^52: the mantissa holds round(w)
  return x == r.top ? 1ull << 40 : (uint64_t)__double_as_longlong(m) & 0xfffffffffffffull;
}

template <int NB>
__device__ __forceinline__ int sm_bin(float x, const SmRow& r) {
  // monotone in x; equal values of the maximum (infinite ones too: NaN converts to 0) give bin 0
  const float d = fmaf(x, -0.5f, r.half_top) * r.bin_scale;
  return (int)min(__float2uint_rz(d), (unsigned)(NB - 1));
}

template <int THREADS, int NB>
struct SmShared {
  static constexpr int kWarps = THREADS / 32, kCap = THREADS < 256 ? THREADS : 256;
  uint32_t lo[NB], hi[NB], cnt[NB];         // this CTA's histogram (mass in two words, number)
  uint64_t m0[NB], m1[NB];                  // the cluster's: over logits, over places
  uint32_t c0[NB], c1[NB];
  uint64_t list[kCap];
  uint64_t wsum[kWarps], wmass[kWarps];
  uint32_t wcnt[kWarps];
  float wmax[kWarps];
  float part_max;
  uint64_t part_lo, part_hi;
  uint64_t above_mass, out_place, out_mass;
  uint32_t above_cnt, bin_cnt, nlist;
  int bin;
  uint64_t total, before;
  int owner;
};

template <typename T, int THREADS, int NB, bool RES>
struct Sampler {
  using S = SmShared<THREADS, NB>;
  using V = SmVec<T>;
  static constexpr int W = THREADS / 32;
  S& s;
  cg::cluster_group cluster;
  int C, rank;
  const T* row;                             // the whole row
  const uint4* data;                        // RES: the slice in shared memory, 16-byte vectors
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

  // Vector v of the slice; values outside the row are -inf.
  __device__ __forceinline__ void load(int v, float (&x)[V::N]) const {
    if constexpr (RES) {
      V::get(data[v], x);
    } else {
#pragma unroll
      for (int j = 0; j < V::N; ++j) {
        const int e = v * V::N + j;
        x[j] = e < len ? sm_ld(row + first + e) : -CUDART_INF_F;
      }
    }
  }
  __device__ __forceinline__ uint32_t index(int v, int j) const {
    return (uint32_t)(first + v * V::N + j - phase);
  }
  // f(value, index) for every value of the slice, each warp its own contiguous part.
  template <typename F>
  __device__ __forceinline__ void each(F f) {
    const int v1 = min(nvec, (warp + 1) * vpw);
    for (int v = warp * vpw + lane; v < v1; v += 32) {
      float x[V::N];
      load(v, x);
#pragma unroll
      for (int j = 0; j < V::N; ++j) f(x[j], index(v, j));
    }
  }

  __device__ __forceinline__ void clear() {
    for (int b = threadIdx.x; b < NB; b += THREADS) s.lo[b] = s.hi[b] = s.cnt[b] = 0u;
    __syncthreads();
  }
  __device__ __forceinline__ void add(int b, float x, bool mass, bool count) {
    if (count) atomicAdd(&s.cnt[b], 1u);
    if (mass) {
      const uint64_t w = sm_weight(x, r);
      const uint32_t l = (uint32_t)w, old = atomicAdd(&s.lo[b], l);
      const uint32_t h = (uint32_t)(w >> 32) + (old + l < old ? 1u : 0u);
      if (h) atomicAdd(&s.hi[b], h);
    }
  }
  // The cluster's histogram in every CTA.
  __device__ void exchange(uint64_t* m, uint32_t* c) {
    sync();
    const int seg = NB / C;
    for (int i = threadIdx.x; i < seg; i += THREADS) {
      const int b = rank * seg + i;
      uint64_t mass = 0;
      uint32_t count = 0;
      for (int q = 0; q < C; ++q) {
        mass += (uint64_t)*at(&s.hi[b], q) << 32;
        mass += *at(&s.lo[b], q);
        count += *at(&s.cnt[b], q);
      }
      for (int q = 0; q < C; ++q) {
        *at(&m[b], q) = mass;
        *at(&c[b], q) = count;
      }
    }
    sync();
  }
  // First bin at which the running number reaches k, or the running mass reaches need; the sums
  // before it go on top of above_mass / above_cnt.
  __device__ void pick(const uint64_t* m, const uint32_t* c, bool by_count, uint32_t k, double need,
                       uint64_t above_mass, uint32_t above_cnt) {
    constexpr int PER = NB / THREADS;
    uint64_t mass[PER], msum = 0;
    uint32_t cnt[PER], csum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      mass[i] = m[threadIdx.x * PER + i], cnt[i] = c[threadIdx.x * PER + i];
      msum += mass[i], csum += cnt[i];
    }
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
    if (threadIdx.x == 0) s.bin = NB - 1, s.bin_cnt = 0, s.above_mass = above_mass, s.above_cnt = above_cnt;
    __syncthreads();
    for (int q = 0; q < W; ++q)
      if (q < warp) mi += s.wmass[q], ci += s.wcnt[q];
    uint64_t run_m = above_mass + mi - msum;
    uint32_t run_c = above_cnt + ci - csum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool was = by_count ? run_c >= k : (double)run_m >= need;
      const uint64_t nm = run_m + mass[i];
      const uint32_t nc = run_c + cnt[i];
      const bool is = by_count ? nc >= k : (double)nm >= need;
      if (!was && is) {
        s.bin = threadIdx.x * PER + i;
        s.bin_cnt = cnt[i];
        s.above_mass = run_m;
        s.above_cnt = run_c;
      }
      run_m = nm, run_c = nc;
    }
    __syncthreads();
  }

  // The place of the last token that the truncation keeps and the mass through it.  Level 0's
  // histogram (m0, c0) is there.
  __device__ void find(bool by_count, uint32_t k, double need, bool mass, uint64_t whole,
                       uint64_t* place, uint64_t* through) {
    pick(s.m0, s.c0, by_count, k, need, 0ull, 0u);
    int bin = s.bin;
    if (bin == NB - 1) {                    // all of any weight is kept
      *place = kSmAll, *through = whole;
      __syncthreads();
      return;
    }
    uint64_t above = s.above_mass;
    uint32_t above_cnt = s.above_cnt, n = s.bin_cnt;
    uint64_t lo = 0, hi = 0;
    const int bin0 = bin;
    for (int level = 0;; ++level) {
      auto member = [&](float x, uint32_t i) {
        if (level == 0) return sm_bin<NB>(x, r) == bin0;
        const uint64_t c = sm_place(x, i);
        return c >= lo && c <= hi;
      };
      if (n <= (uint32_t)S::kCap) {
        // few: collect them in CTA 0, rank them, add their weights in order
        if (threadIdx.x == 0) s.nlist = 0;
        sync();
        each([&](float x, uint32_t i) {
          if (member(x, i)) {
            const uint32_t j = atomicAdd(at(&s.nlist, 0), 1u);
            if (j < (uint32_t)S::kCap) *at(&s.list[j], 0) = sm_place(x, i);
          }
        });
        sync();
        if (rank == 0) {
          const int t = threadIdx.x;
          uint64_t mine = kSmAll;
          int at_rank = 0;
          if (t < (int)n) {
            mine = s.list[t];
            for (uint32_t j = 0; j < n; ++j) at_rank += s.list[j] < mine;
          }
          __syncthreads();
          if (t < (int)n) s.list[at_rank] = mine;
          __syncthreads();
          mine = t < (int)n ? s.list[t] : kSmAll;
          const uint64_t w = mass && t < (int)n ? sm_weight(sm_place_value(mine), r) : 0ull;
          uint64_t run = w;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint64_t a = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += a;
          }
          const uint64_t ws = __shfl_sync(0xffffffffu, run, 31);
          if (lane == 0) s.wmass[warp] = ws;
          __syncthreads();
          for (int q = 0; q < W; ++q)
            if (q < warp) run += s.wmass[q];
          run += above;
          if (t < (int)n) {
            const bool is = by_count ? above_cnt + t + 1 == k : (double)run >= need;
            const bool was = !by_count && (double)(run - w) >= need;
            if (is && !was)
              for (int q = 0; q < C; ++q) *at(&s.out_place, q) = mine, *at(&s.out_mass, q) = run;
          }
        }
        sync();
        *place = s.out_place, *through = s.out_mass;
        return;
      }
      if (level == 0) {                     // the range of places in the bin
        uint64_t a = kSmAll, b = 0;
        each([&](float x, uint32_t i) {
          if (sm_bin<NB>(x, r) == bin0) {
            const uint64_t c = sm_place(x, i);
            a = min(a, c), b = max(b, c);
          }
        });
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
      int shift = 64 - __clzll((long long)(hi - lo)) - (31 - __clz(NB));
      shift = max(shift, 0);
      clear();
      each([&](float x, uint32_t i) {
        if (level == 0 && sm_bin<NB>(x, r) != bin0) return;
        const uint64_t c = sm_place(x, i);
        if (c >= lo && c <= hi) add((int)((c - lo) >> shift), x, mass, true);
      });
      exchange(s.m1, s.c1);
      pick(s.m1, s.c1, by_count, k, need, above, above_cnt);
      bin = s.bin, n = s.bin_cnt, above = s.above_mass, above_cnt = s.above_cnt;
      lo += (uint64_t)bin << shift;
      hi = lo + min(hi - lo, (uint64_t)((1ull << shift) - 1));
      __syncthreads();
    }
  }
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

template <typename T, int THREADS, int NB, bool RES>
__global__ void __launch_bounds__(THREADS) sample_kernel(const SmArgs a) {
  using Sm = Sampler<T, THREADS, NB, RES>;
  using Vv = SmVec<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  SmShared<THREADS, NB>& s = *reinterpret_cast<SmShared<THREADS, NB>*>(smem);
  constexpr size_t kData = (sizeof(SmShared<THREADS, NB>) + 15) / 16 * 16;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t rw = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* row = static_cast<const T*>(a.logits) + rw * a.ld;
  const float t = a.temperature ? a.temperature[rw] : 1.f;
  const float p = a.top_p ? a.top_p[rw] : 1.f;
  const float mp = a.min_p ? a.min_p[rw] : 0.f;
  const double un = a.u[rw];
  const int k = a.top_k ? a.top_k[rw] : 0;
  const bool bad = !(t >= 0.f && t < CUDART_INF_F && p > 0.f && p <= 1.f && mp >= 0.f && mp <= 1.f &&
                     un >= 0.0 && un < 1.0);
  if (bad) {
    if (rank == 0 && tid == 0) {
      a.ids[rw] = -1;
      if (a.prob) a.prob[rw] = CUDART_NAN_F;
    }
    return;
  }
  const int first = min(rank * a.slice, a.V), len = min(a.slice, a.V - first);
  const T* src = row + first;
  uint4* data = reinterpret_cast<uint4*>(smem + kData);
  const int phase = RES ? (int)((uintptr_t)src % 16 / sizeof(T)) : 0;
  const int nvec = len > 0 ? (phase + len + Vv::N - 1) / Vv::N : 0;
  Sm z = {s, cluster, C, rank, row, data, first, len, phase, nvec, (nvec + Sm::W - 1) / Sm::W,
          lane, warp, {}};

  // the slice to shared memory, and its maximum (NaN when it holds one)
  float best = -CUDART_INF_F;
  if constexpr (RES) {
    const uint4* g = reinterpret_cast<const uint4*>(src - phase);
    for (int v0 = tid; v0 < nvec; v0 += THREADS * 8) {
      uint4 q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int v = v0 + i * THREADS;
        if (v < nvec) {
          if (v * Vv::N >= phase && (v + 1) * Vv::N <= phase + len) {
            q[i] = __ldcs(g + v);
          } else {                          // the ragged ends of the slice
            T e[Vv::N];
            uint4 w = make_uint4(Vv::kMinusInf, Vv::kMinusInf, Vv::kMinusInf, Vv::kMinusInf);
            memcpy(e, &w, 16);
#pragma unroll
            for (int j = 0; j < Vv::N; ++j) {
              const int at = v * Vv::N + j - phase;
              if (at >= 0 && at < len) e[j] = src[at];
            }
            memcpy(&w, e, 16);
            q[i] = w;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int v = v0 + i * THREADS;
        if (v < nvec) {
          float x[Vv::N];
          Vv::get(q[i], x);
#pragma unroll
          for (int j = 0; j < Vv::N; ++j) best = sm_max_nan(best, x[j]);
          data[v] = q[i];
        }
      }
    }
  } else {
    z.each([&](float x, uint32_t) { best = sm_max_nan(best, x); });
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = sm_max_nan(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) s.wmax[warp] = best;
  __syncthreads();
  if (tid == 0) {
    for (int q = 0; q < Sm::W; ++q) best = sm_max_nan(best, s.wmax[q]);
    s.part_max = best;
  }
  z.sync();
  float top = -CUDART_INF_F;
  for (int q = 0; q < C; ++q) top = sm_max_nan(top, *z.at(&s.part_max, q));
  if (isnan(top) || top == -CUDART_INF_F) {
    if (rank == 0 && tid == 0) {
      a.ids[rw] = -1;
      if (a.prob) a.prob[rw] = isnan(top) ? CUDART_NAN_F : 0.f;
    }
    z.sync();                               // the others may still read this CTA's maximum
    return;
  }
  z.r.top = top;
  z.r.half_top = 0.5f * top;
  z.r.bin_scale = 2.f * (NB - 1) / 28.5f / t;
  z.r.topd = (double)top;
  z.r.c = t > 0.f ? 1.4426950408889634 / (double)t : 0.0;
  const SmRow r = z.r;

  // the border: place of the last kept token
  uint64_t border = kSmAll;
  if (t == 0.f) {
    border = sm_place(top, 0xffffffffu);
  } else {
    const bool by_k = k > 0 && k < a.V, by_p = p < 1.f;
    if (by_k || by_p) {
      z.clear();
      z.each([&](float x, uint32_t) {
        const int b = sm_bin<NB>(x, r);
        if (b < NB - 1) z.add(b, x, by_p, by_k || by_p);
      });
      z.exchange(s.m0, s.c0);
      uint64_t whole = 0;
      if (by_p) {
        uint64_t m = 0;
        for (int b = tid; b < NB; b += THREADS) m += s.m0[b];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
        if (lane == 0) s.wsum[warp] = m;
        __syncthreads();
        for (int q = 0; q < Sm::W; ++q) whole += s.wsum[q];
        __syncthreads();
      }
      if (by_k) z.find(true, (uint32_t)k, 0.0, by_p, whole, &border, &whole);
      if (by_p) {
        uint64_t through;
        z.find(false, 0u, (double)p * (double)whole, true, whole, &border, &through);
      }
    }
    if (mp > 0.f) {
      // the smallest logit with (x - top) / T >= log(min_p): bisection over keys, at first round
      // the nearest float to top + T log(min_p)
      const double cut = log((double)mp) * 1.4426950408889634;
      auto in = [&](uint32_t key) {
        const float x = sm_value(key);
        return x == top || ((double)x - (double)top) * r.c >= cut;
      };
      const uint32_t lowest = 0x007fffffu, top_key = sm_key(top);   // key of -inf: never in
      const uint32_t guess = sm_key((float)fmax((double)top + cut / r.c, -3.4e38));
      uint32_t lo = guess > lowest + 4 && !in(guess - 4) ? guess - 4 : lowest;
      uint32_t hi = guess < top_key - 4 && in(guess + 4) ? guess + 4 : top_key;
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (in(mid)) hi = mid;
        else lo = mid;
      }
      border = min(border, (uint64_t)(~hi) << 32 | 0xffffffffu);
    }
  }
  const float xb = border == kSmAll ? -CUDART_INF_F : sm_place_value(border);
  const uint32_t ib = (uint32_t)border;
  auto weight = [&](float x, uint32_t i) -> uint64_t {
    if (x > xb || (x == xb && i <= ib)) {
      if (sm_bin<NB>(x, r) < NB - 1) return sm_weight(x, r);
    }
    return 0ull;
  };
  uint64_t mass = 0;
  z.each([&](float x, uint32_t i) { mass += weight(x, i); });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  if (lane == 0) s.wsum[warp] = mass;
  z.sync();
  // the warp whose part holds the target
  if (tid < 32) {
    uint64_t total = 0;
    const int n = C * Sm::W;
    for (int q0 = 0; q0 < n; q0 += 32) {
      const int q = q0 + lane;
      uint64_t w = q < n ? *z.at(&s.wsum[q % Sm::W], q / Sm::W) : 0ull;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      total += w;
    }
    const uint64_t target = t == 0.f ? 0ull : min((uint64_t)(un * (double)total), total - 1);
    uint64_t run = 0;
    for (int q0 = 0; q0 < n; q0 += 32) {
      const int q = q0 + lane;
      const uint64_t w = q < n ? *z.at(&s.wsum[q % Sm::W], q / Sm::W) : 0ull;
      uint64_t inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t b = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += b;
      }
      const uint64_t end = run + inc, start = end - w;
      if (w > 0 && end > target && start <= target) {
        s.owner = q;
        s.before = target - start;          // weight to pass inside the part
        s.total = total;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  if (C > 1) cluster.sync();                // no CTA leaves while its sums may be read
  if (s.owner != rank * Sm::W + warp) return;
  uint64_t target = s.before, run = 0;
  const int v1 = min(nvec, (warp + 1) * z.vpw);
  for (int v0 = warp * z.vpw; v0 < v1; v0 += 32) {
    const int v = v0 + lane;
    float x[Vv::N];
    uint64_t w[Vv::N], sum = 0;
    if (v < v1) {
      z.load(v, x);
#pragma unroll
      for (int j = 0; j < Vv::N; ++j) w[j] = weight(x[j], z.index(v, j)), sum += w[j];
    }
    uint64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t b = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += b;
    }
    uint64_t at = run + inc - sum;
    if (sum > 0 && at <= target && at + sum > target) {
#pragma unroll
      for (int j = 0; j < Vv::N; ++j) {
        if (at <= target && at + w[j] > target) {
          a.ids[rw] = (int32_t)z.index(v, j);
          if (a.prob)
            a.prob[rw] = t == 0.f ? 1.f
                         : (float)((x[j] == top ? 1.0 : exp(((double)x[j] - (double)top) / (double)t)) *
                                   kSmOne / (double)s.total);
        }
        at += w[j];
      }
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
    if (run > target) break;
  }
}

template <typename T, int THREADS, int NB, bool RES>
cudaError_t sm_launch(const SmArgs& a, int64_t rows, int C, size_t smem, cudaStream_t st) {
  auto* k = sample_kernel<T, THREADS, NB, RES>;
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
  constexpr int kSmall = 128, kSmallBins = 256, kLarge = 512, kBins = 1024;
  constexpr size_t kFixedSmall = (sizeof(SmShared<kSmall, kSmallBins>) + 15) / 16 * 16;
  constexpr size_t kFixed = (sizeof(SmShared<kLarge, kBins>) + 15) / 16 * 16;
  constexpr size_t kHalf = 113 * 1024, kFull = 227 * 1024;   // two CTAs a SM, one CTA a SM
  const auto bytes = [&](int C) { return ((size_t)((a.V + C - 1) / C) * sizeof(T) + 31) / 16 * 16; };
  if (a.V <= 4096) {
    a.slice = a.V;
    return sm_launch<T, kSmall, kSmallBins, true>(a, rows, 1, kFixedSmall + bytes(1), st);
  }
  // as many CTAs a row as its slices need to lie two to a SM; more while the rows leave SMs idle
  int C = 1;
  while (C < 8 && (kFixed + bytes(C) > kHalf || (rows * C < 2 * sms && a.V / C > 4096))) C *= 2;
  a.slice = (a.V + C - 1) / C;
  if (rows * C > INT32_MAX) return cudaErrorInvalidValue;
  if (kFixed + bytes(C) <= kFull)
    return sm_launch<T, kLarge, kBins, true>(a, rows, C, kFixed + bytes(C), st);
  return sm_launch<T, kLarge, kBins, false>(a, rows, C, kFixed, st);
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
