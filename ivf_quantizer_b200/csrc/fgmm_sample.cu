// One draw per row of scores from its truncated softmax (temperature, top-k, top-p, min-p) with
// given uniforms.  The definition is that of fgmm_sample_logits in include/fgmm.h.
//
// Weights are 64-bit integers, w_i = round(2^40 exp((l_i - max l) / T)), so every sum is exact and
// independent of its order: the draw is reproducible, and ties of equal logits are exact.
// 2^40 leaves 2^22 tokens room in 63 bits; the error of a sum of n weights is at most n / 2 units.
//
// The tokens that top-k and top-p keep are a prefix of the order (logit descending, index
// ascending), so a truncation is a pair (border key, number of tokens kept at the border key).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "fgmm_internal.h"

namespace fgmm {
namespace {

constexpr int kSmThreads = 1024;
constexpr double kSmOne = 1099511627776.0;  // 2^40

__device__ __forceinline__ float sm_ld(const float* p) { return __ldg(p); }
__device__ __forceinline__ float sm_ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Order-preserving integer of a logit; -0 and +0 are one value.
__device__ __forceinline__ uint32_t sm_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float sm_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ uint64_t sm_weight(float x, float top, double inv_t) {
  if (x == top) return 1ull << 40;
  return (uint64_t)__double2ull_rn(exp(((double)x - (double)top) * inv_t) * kSmOne);
}

struct SmSum {
  uint64_t mass;
  uint32_t count;
};

// Block-wide sum; every thread receives it.
__device__ SmSum sm_block_sum(uint64_t mass, uint32_t count, uint64_t* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mass += __shfl_xor_sync(0xffffffffu, mass, o);
    count += __shfl_xor_sync(0xffffffffu, count, o);
  }
  uint32_t* shc = reinterpret_cast<uint32_t*>(sh + 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh[threadIdx.x >> 5] = mass;
    shc[threadIdx.x >> 5] = count;
  }
  __syncthreads();
  SmSum r = {0, 0};
  for (int w = 0; w < kSmThreads / 32; ++w) r.mass += sh[w], r.count += shc[w];
  return r;
}

// Weight and number of the tokens whose key is at least `key`.
template <typename T>
__device__ SmSum sm_at_least(const T* row, int V, uint32_t key, float top, double inv_t,
                             bool want_mass, uint64_t* sh) {
  uint64_t mass = 0;
  uint32_t count = 0;
  for (int i = threadIdx.x; i < V; i += kSmThreads) {
    const float x = sm_ld(row + i);
    if (sm_key(x) >= key) {
      ++count;
      if (want_mass) mass += sm_weight(x, top, inv_t);
    }
  }
  return sm_block_sum(mass, count, sh);
}

template <typename T>
__global__ void __launch_bounds__(kSmThreads)
    sample_kernel(const T* __restrict__ logits, int V, int64_t ld, const float* temperature,
                  const int32_t* top_k, const float* top_p, const float* min_p, const double* u,
                  int32_t* ids, float* prob) {
  __shared__ uint64_t sh[64];
  __shared__ uint32_t s_top;
  __shared__ int s_bad, s_first;
  const int64_t r = blockIdx.x;
  const T* row = logits + r * ld;
  const int tid = threadIdx.x;
  const float t = temperature ? temperature[r] : 1.f;
  const float p = top_p ? top_p[r] : 1.f;
  const float mp = min_p ? min_p[r] : 0.f;
  const double un = u[r];
  const int k = top_k ? top_k[r] : 0;
  if (tid == 0) {
    s_top = 0u;
    s_first = INT32_MAX;
    s_bad = !(t >= 0.f && t < CUDART_INF_F && p > 0.f && p <= 1.f && mp >= 0.f && mp <= 1.f &&
              un >= 0.0 && un < 1.0);
  }
  __syncthreads();
  uint32_t best = 0u;
  bool nan = false;
  for (int i = tid; i < V; i += kSmThreads) {
    const float x = sm_ld(row + i);
    nan |= isnan(x);
    best = max(best, sm_key(x));
  }
  atomicMax(&s_top, best);
  if (nan) s_bad = 1;
  __syncthreads();
  const uint32_t top_key = s_top;
  const float top = sm_value(top_key);
  if (s_bad || top == -CUDART_INF_F) {
    if (tid == 0) {
      ids[r] = -1;
      if (prob) prob[r] = s_bad ? CUDART_NAN_F : 0.f;
    }
    return;
  }
  if (t == 0.f) {
    for (int i = tid; i < V; i += kSmThreads)
      if (sm_key(sm_ld(row + i)) == top_key) {
        atomicMin(&s_first, i);
        break;
      }
    __syncthreads();
    if (tid == 0) {
      ids[r] = s_first;
      if (prob) prob[r] = 1.f;
    }
    return;
  }
  const double inv_t = 1.0 / (double)t;
  // border: tokens above `border`, and the first `ties` tokens at it
  uint32_t border = 0u, ties = UINT32_MAX;
  uint64_t whole = 0;
  if (k > 0 && k < V) {
    uint32_t lo = 0u, hi = top_key;             // count(>= lo) >= k; the largest such key
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      if (sm_at_least(row, V, mid, top, inv_t, false, sh).count >= (uint32_t)k) lo = mid;
      else hi = mid - 1;
    }
    border = lo;
    const SmSum above = border == UINT32_MAX
                            ? SmSum{0, 0}
                            : sm_at_least(row, V, border + 1, top, inv_t, true, sh);
    ties = (uint32_t)k - above.count;
    whole = above.mass + ties * sm_weight(sm_value(border), top, inv_t);
  } else if (p < 1.f) {
    whole = sm_at_least(row, V, 0u, top, inv_t, true, sh).mass;
  }
  if (p < 1.f) {
    const double need = (double)p * (double)whole;
    uint32_t lo = border, hi = top_key;         // mass(>= lo) >= need; the largest such key
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      if ((double)sm_at_least(row, V, mid, top, inv_t, true, sh).mass >= need) lo = mid;
      else hi = mid - 1;
    }
    const uint64_t above =
        lo == top_key ? 0ull : sm_at_least(row, V, lo + 1, top, inv_t, true, sh).mass;
    const uint64_t w = sm_weight(sm_value(lo), top, inv_t);
    const uint32_t most = lo == border ? ties : UINT32_MAX;
    uint32_t j = 1;                             // the j-th tie stays while the weight before it is short
    if (w > 0) {
      uint32_t a = 1, b = min(most, (uint32_t)V);
      while (a < b) {                           // smallest j with above + j w >= need
        const uint32_t mid = a + (b - a) / 2;
        if ((double)(above + mid * w) >= need) b = mid;
        else a = mid + 1;
      }
      j = a;
    } else {
      j = most;
    }
    border = lo;
    ties = j;
  }
  const double floor_t = mp > 0.f ? log((double)mp) : -CUDART_INF;
  auto kept_value = [&](float x) {
    return x == top || ((double)x - (double)top) * inv_t >= floor_t;
  };
  uint64_t mass = 0;
  for (int i = tid; i < V; i += kSmThreads) {
    const float x = sm_ld(row + i);
    if (sm_key(x) > border && kept_value(x)) mass += sm_weight(x, top, inv_t);
  }
  uint64_t total = sm_block_sum(mass, 0, sh).mass;
  const uint64_t wb = kept_value(sm_value(border)) ? sm_weight(sm_value(border), top, inv_t) : 0ull;
  uint64_t ntie = 0;
  if (wb) {
    const uint32_t lo = sm_at_least(row, V, border, top, inv_t, false, sh).count;
    const uint32_t hi = border == UINT32_MAX
                            ? 0u
                            : sm_at_least(row, V, border + 1, top, inv_t, false, sh).count;
    ntie = min(lo - hi, ties);
  }
  total += ntie * wb;
  const uint64_t target = min((uint64_t)(un * (double)total), total - 1);
  // the draw: chunks of one token a thread, in index order
  uint64_t run = 0;
  uint32_t seen = 0;
  for (int i0 = 0; i0 < V; i0 += kSmThreads) {
    const int i = i0 + tid;
    const float x = i < V ? sm_ld(row + i) : -CUDART_INF_F;
    const bool in = i < V;
    const bool tie = in && sm_key(x) == border;
    uint64_t w = in && sm_key(x) > border && kept_value(x) ? sm_weight(x, top, inv_t) : 0ull;
    // inclusive scans of ties, then of weights
    uint32_t c = tie;
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += y;
    }
    uint32_t* shc = reinterpret_cast<uint32_t*>(sh + 32);
    __syncthreads();
    const uint32_t cw = __shfl_sync(0xffffffffu, c, 31);
    if (lane == 0) shc[warp] = cw;
    __syncthreads();
    uint32_t call = 0;
    for (int q = 0; q < kSmThreads / 32; ++q) {
      if (q < warp) c += shc[q];
      call += shc[q];
    }
    if (tie && seen + c <= ties) w = wb;
    uint64_t s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    const uint64_t sw = __shfl_sync(0xffffffffu, s, 31);
    if (lane == 0) sh[warp] = sw;
    __syncthreads();
    uint64_t sall = 0;
    for (int q = 0; q < kSmThreads / 32; ++q) {
      if (q < warp) s += sh[q];
      sall += sh[q];
    }
    if (w > 0 && run + s > target && run + s - w <= target) {
      ids[r] = i;
      if (prob)
        prob[r] = (float)(x == top ? kSmOne / (double)total
                                   : exp(((double)x - (double)top) * inv_t) * kSmOne / (double)total);
    }
    run += sall;
    seen += call;
    if (run > target) break;
  }
}

}  // namespace

// ------------------------------------------------------------------ launcher
cudaError_t launch_sample_logits(const void* logits, int dtype, int64_t rows, int V, int64_t ld,
                                 const float* temperature, const int32_t* top_k,
                                 const float* top_p, const float* min_p, const double* u,
                                 int32_t* ids, float* prob, cudaStream_t s) {
  if (dtype == FGMM_F32)
    sample_kernel<float><<<(unsigned)rows, kSmThreads, 0, s>>>(
        static_cast<const float*>(logits), V, ld, temperature, top_k, top_p, min_p, u, ids, prob);
  else
    sample_kernel<__nv_bfloat16><<<(unsigned)rows, kSmThreads, 0, s>>>(
        static_cast<const __nv_bfloat16*>(logits), V, ld, temperature, top_k, top_p, min_p, u, ids,
        prob);
  return cudaGetLastError();
}

}  // namespace fgmm
