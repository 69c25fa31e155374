// 4-bit codes of vectors (OCP Microscaling Formats v1.0, MXFP4: blocks of 32 e2m1 codes with
// one e8m0 scale) and the scores of queries against them.  The layout of codes and scales is
// that of include/fgmm.h.
//
//   encode  reads 4 (or 2) bytes a value, writes 17/32: bound by reading
//   decode  the reverse: bound by writing
//   scores  out = alpha Q X^T + bias over the decoded values
#include <cuda_bf16.h>

#include <type_traits>

#include "fgmm_internal.h"
#include "mxf4_ptx.cuh"

namespace fgmm {
namespace {

// The word that fgmm_mx4_status_word gives out.  A variable of the module: there before the first
// call, whatever captures or allocates at that time, and the same for every thread.
__device__ int mx_status_word = FGMM_OK;

constexpr int kMxThreads = 256;

__device__ __forceinline__ float mx_ld(const float* p) { return __ldg(p); }
__device__ __forceinline__ float mx_ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void mx_st(float* p, float v) { *p = v; }
__device__ __forceinline__ void mx_st(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four values, already scaled, to four e2m1 codes (nearest, ties to even, saturating).
__device__ __forceinline__ uint32_t mx_codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b, a, b};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r & 0xffffu;
}
// Value of the code in the low four bits.  The three magnitude bits (two of exponent, bias 1, one of
// mantissa) placed at the top of a float's mantissa and the bottom of its exponent read as the value
// times 2^-126, the subnormal 0.5 included.
__device__ __forceinline__ float mx_value(uint32_t b) {
  return __uint_as_float((b & 7u) << 22 | (b & 8u) << 28) * 8.507059173023462e37f;  // 2^126
}
// The value of an e8m0 scale byte.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return s == 255u ? __int_as_float(0x7fc00000)
                   : (s == 0u ? __int_as_float(0x00400000) : __int_as_float((int)(s << 23)));
}

// Pieces of 32 bytes of a row: what a thread encodes or decodes at once.
template <typename T>
struct MxPiece;
template <>
struct MxPiece<float> {
  static constexpr int N = 8;
  using Codes = uint32_t;
  // the piece's largest magnitude as the bits of a float (NaN and infinity sort above the finite)
  static __device__ __forceinline__ uint32_t top(const uint32_t (&w)[8]) {
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max(a, w[j] & 0x7fffffffu);
    return a;
  }
  static __device__ __forceinline__ float at(const uint32_t (&w)[8], int j) { return __uint_as_float(w[j]); }
  static __device__ __forceinline__ void put(uint32_t (&w)[8], int j, float v) { w[j] = __float_as_uint(v); }
};
template <>
struct MxPiece<__nv_bfloat16> {
  static constexpr int N = 16;
  using Codes = uint64_t;
  static __device__ __forceinline__ uint32_t top(const uint32_t (&w)[8]) {
    uint32_t a = 0;                         // both halves of a word at once
#pragma unroll
    for (int j = 0; j < 8; ++j) a = __vmaxu2(a, w[j] & 0x7fff7fffu);
    return max(a << 16, a & 0xffff0000u);
  }
  static __device__ __forceinline__ float at(const uint32_t (&w)[8], int j) {
    return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
  }
  static __device__ __forceinline__ void put(uint32_t (&w)[8], int j, float v) {
    const uint32_t b = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    if (j & 1) w[j >> 1] |= b << 16;
    else w[j >> 1] = b;
  }
};

// The pieces of a thread: piece i of the padded rows (nb blocks each) with stride `step`.
struct MxPieces {
  int64_t i, row, drow, step;
  int seg, dseg, segs;
  __device__ __forceinline__ MxPieces(int segs_) : segs(segs_) {
    i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
    step = (int64_t)gridDim.x * kMxThreads;
    row = i / segs, seg = (int)(i - row * segs);
    drow = step / segs, dseg = (int)(step - drow * segs);
  }
  __device__ __forceinline__ void next() {
    i += step, row += drow, seg += dseg;
    if (seg >= segs) seg -= segs, ++row;
  }
};
__device__ __forceinline__ int64_t mx_scale_at(int64_t row, int b, int nkc) {
  return ((row >> 7) * nkc + (b >> 2)) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4 + (b & 3);
}

// 32 bytes (p aligned to them) that are not read again.
__device__ __forceinline__ void mx_ld32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

__device__ __forceinline__ void mx_st32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A thread encodes 32 bytes of a row at a time, four (fp32) or two (bf16) neighbouring lanes a block;
// codes lie in the order of the threads, so a warp writes them as one contiguous piece.  Two pieces a
// thread are loaded before either is used.  Bound by memory; a lane a 4 values took
// 1266 us at 10^6 x 960 bf16 (issue).  BYTES: what rows allow to load at once
// (bf16 x 960 by 8 and 4 bytes, row strides 964 and 962, 469 and 523 us; by single values both 890).
//
// TILES: the rows are walked as if padded to whole scale tiles (4 blocks), so that four scales, the
// padding included, leave as one word; lanes behind the last block idle.  10^6 rows, without and with,
// us: fp32 x 128 100 and 91, x 448 350 and 325, x 960 762 and 690, bf16 x 512 225 and 213, x 960 443
// and 423; but fp32 x 96 (a quarter idle) 80 and 89, bf16 x 160 91 and 113.  (32 bytes at once
// against twice 16: 345 and 375 at fp32 x 512, no difference in bf16.)
template <typename T, int BYTES, bool TILES>
__global__ void __launch_bounds__(kMxThreads, TILES ? 6 : 1)
    mx4_encode_kernel(const T* __restrict__ X, int64_t n, int D, int64_t ldx, int nb, int nkc,
                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  using P = MxPiece<T>;
  constexpr int LB = 32 / P::N, U = 2;      // lanes a block, pieces in flight
  ptx::grid_release();                      // (kernels that read these codes may set themselves up)
  MxPieces p((TILES ? 4 * nkc : nb) * LB);
  const int64_t rows = (n + 127) / 128 * 128;   // rows behind the last only have scales, 0
  // (whole warps stay together for the exchange: a warp leaves when its first piece is behind the end)
  const int64_t pieces = rows * p.segs;
  while (p.i - (threadIdx.x & 31) < pieces) {
    uint32_t w[U][8];
    int64_t at[U], row[U];
    int seg[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = TILES ? p.row * (nb * LB) + p.seg : p.i;
      row[u] = p.row, seg[u] = p.seg;
      p.next();
      const int d = seg[u] * P::N;
      const T* x = X + row[u] * ldx + d;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[u][j] = 0u;
      if (row[u] < n) {
        if (BYTES > (int)sizeof(T) && d + P::N <= D) {
          if constexpr (BYTES == 32) {
            mx_ld32(x, w[u]);
          } else if constexpr (BYTES < 16) {        // (cached: the same lines are read several times)
#pragma unroll
            for (int j = 0; j < 8; j += BYTES / 4) {
              if constexpr (BYTES == 8) {
                const uint2 a = __ldg(reinterpret_cast<const uint2*>(x) + j / 2);
                w[u][j] = a.x, w[u][j + 1] = a.y;
              } else {
                w[u][j] = __ldg(reinterpret_cast<const uint32_t*>(x) + j);
              }
            }
          } else {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(x));
            const uint4 b = __ldcs(reinterpret_cast<const uint4*>(x) + 1);
            w[u][0] = a.x, w[u][1] = a.y, w[u][2] = a.z, w[u][3] = a.w;
            w[u][4] = b.x, w[u][5] = b.y, w[u][6] = b.z, w[u][7] = b.w;
          }
        } else if (!TILES || d < D) {
#pragma unroll
          for (int j = 0; j < P::N; ++j)
            if (d + j < D) P::put(w[u], j, mx_ld(x + j));
            else if (j % 2 == 0 || P::N == 8) P::put(w[u], j, 0.f);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t a = P::top(w[u]);
#pragma unroll
      for (int o = 1; o < LB; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
      const uint32_t e = a >> 23;
      const bool bad = e == 255u;
      const uint32_t s = bad ? 255u : e > 2u ? e - 2u : 0u;   // floor(log2 a) - 2 + 127, at least 0
      const float inv = __uint_as_float((bad ? 0u : 254u - s) << 23);
      typename P::Codes c = 0;
#pragma unroll
      for (int j = 0; j < P::N; j += 4)
        c |= (typename P::Codes)mx_codes4(P::at(w[u], j) * inv, P::at(w[u], j + 1) * inv,
                                          P::at(w[u], j + 2) * inv, P::at(w[u], j + 3) * inv)
             << (4 * j);
      if (bad) c = 0;
      uint32_t four = s;                    // TILES: the scales of four blocks, in the lanes of the first
      if constexpr (TILES) {
        four |= __shfl_xor_sync(0xffffffffu, four, LB) << 8;
        four |= __shfl_xor_sync(0xffffffffu, four, 2 * LB) << 16;
      }
      if (row[u] >= rows) continue;
      if (row[u] < n && (!TILES || seg[u] < nb * LB)) reinterpret_cast<typename P::Codes*>(codes)[at[u]] = c;
      const int b = seg[u] / LB;
      if constexpr (TILES) {
        if (seg[u] % (4 * LB) == 0)
          *reinterpret_cast<uint32_t*>(scales + mx_scale_at(row[u], b, nkc)) = four;
      } else if (seg[u] % LB == 0) {
        scales[mx_scale_at(row[u], b, nkc)] = row[u] < n ? (uint8_t)s : 0;
        if (b == nb - 1)                    // and the padding of the last scale tile
          for (int z = nb; z < 4 * nkc; ++z) scales[mx_scale_at(row[u], z, nkc)] = 0;
      }
    }
  }
}

// A thread decodes BYTES of the rows r, r + 32, r + 64, r + 96 of a 128-row tile: the four rows' scales
// of a block lie in the same 16 bytes of the scale tile.  Threads follow one another along a row, then
// to the next one.  Bound by writing.  AT: the bytes that rows allow to store at once.  10^6 rows, us,
// with a warp on 512 bytes of a row, 16 a lane, and so: fp32 x 960 671 and 645, bf16 x 960 447 and 366,
// bf16 x 128 111 and 51.  With the encoder's mapping (a sequence of pieces of consecutive rows) the
// address arithmetic took it to 979 at fp32 x 960.  Rows off a 16-byte boundary by single values, with
// 8 a thread, and so: bf16 x 960 with a row stride of 964 2714 and 510, of 962 522, of 961 1040.
template <typename T, int BYTES, int AT>
__global__ void __launch_bounds__(kMxThreads)
    mx4_decode_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      int64_t n, int D, int nb, int nkc, int segs, int64_t pieces, T* __restrict__ out,
                      int64_t ldo) {
  constexpr int N = BYTES / sizeof(T), WORDS = BYTES / 4;
  using Codes = std::conditional_t<N == 4, uint16_t, std::conditional_t<N == 8, uint32_t, uint64_t>>;
  ptx::grid_wait();
  const int64_t step = (int64_t)gridDim.x * kMxThreads;
  for (int64_t i0 = (int64_t)blockIdx.x * kMxThreads; i0 + threadIdx.x < pieces; i0 += step) {
    const int64_t r0 = i0 / segs;                   // (the block's; the thread's from it by 32 bits)
    const uint32_t at = (uint32_t)(i0 - r0 * segs) + threadIdx.x, dr = at / (uint32_t)segs;
    const int64_t rr = r0 + dr;                     // row tile * 32 + row within the quarter
    const int d = (int)(at - dr * segs) * N;
    const int64_t row0 = (rr >> 5) * 128 + (rr & 31);
    const uint4 sw = __ldg(reinterpret_cast<const uint4*>(
        scales + ((rr >> 5) * nkc + (d >> 7)) * 512 + (rr & 31) * 16));
    const uint32_t words[4] = {sw.x, sw.y, sw.z, sw.w};
    const uint8_t* from = codes + row0 * nb * 16 + (d >> 1);
    Codes c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      c[q] = row0 + 32 * q < n ? __ldcs(reinterpret_cast<const Codes*>(from + (int64_t)32 * q * nb * 16)) : Codes(0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (row0 + 32 * q >= n) break;
      const float s = mx_scale((words[q] >> (d >> 2 & 24)) & 255u);
      T* o = out + (row0 + 32 * q) * ldo + d;
      float v[N];
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = mx_value((uint32_t)(c[q] >> (4 * j))) * s;
      if (AT >= 4 && d + N <= D) {
        uint32_t w[WORDS];
#pragma unroll
        for (int j = 0; j < WORDS; ++j) {
          if constexpr (sizeof(T) == 4) {
            w[j] = __float_as_uint(v[j]);
          } else {                                  // (exact: a code has two significant bits)
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = reinterpret_cast<const uint32_t&>(t);
          }
        }
        if constexpr (AT == 32) {
          mx_st32(o, w);
        } else {
#pragma unroll
          for (int j = 0; j < WORDS; j += AT / 4) {
            uint32_t* to = reinterpret_cast<uint32_t*>(o) + j;
            if constexpr (AT == 16) __stcs(reinterpret_cast<uint4*>(to), make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]));
            else if constexpr (AT == 8) __stcs(reinterpret_cast<uint2*>(to), make_uint2(w[j], w[j + 1]));
            else __stcs(to, w[j]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (d + j < D) mx_st(o + j, v[j]);
      }
    }
  }
}

// ------------------------------------------------------------------ scores (tcgen05)
// The vectors are the M side of the products (128 of them a tile: TMEM lane = vector), the
// queries the N side (NT a tile: TMEM column = query).  The codes then stream through the wide
// side whatever the number of queries, and a warp holds 32 consecutive scores of one query.
//
// A CTA walks its tiles: a producer warp fills a ring of stages (KB bytes of each of 128 vectors and
// their scale tiles), another copies a stage's scales to TMEM and issues its K = 64 block-scaled
// products, and the epilogue warps drain one of two accumulators while the other is filled.  Three
// kernels differ in how a stage is filled:
//   rows longer than 256 dimensions: TMA boxes of 128 vectors x 128 bytes, with the queries' beside;
//   shorter ones: a tile is one contiguous piece of memory, so it comes as a single bulk copy, and
//   two or four warps put it into the swizzled order, while the queries' tile stays in shared memory
//   (one query and 10^6 vectors by boxes and by copies: 30.6 and 19.8 us at 96 dimensions, 29.5 and 17.4
//   at 32, 41.7 and 33.7 at 224);
//   many queries of long rows: pairs of CTAs, further down.
//
// The output is the larger part of the traffic for short rows.  Scores written straight from
// registers are 128-byte pieces that straddle two lines when the row stride is odd (156 us against
// 84 aligned, 1000 x 100003 x 128 fp32), so tiles of 64 queries and more pass through shared memory
// and leave as bulk copies of a query's 128 scores, the ragged ends aside.
constexpr int kMxBM = 128;         // vectors a tile
constexpr int kMxMaxStages = 10;

// What the kernels of one CTA share: the epilogue's side.
template <int NT>
struct MxEpi {
  static constexpr bool kStaged = NT >= 64;
  static constexpr int kWarps = kStaged ? NT / 8 : 4;         // four of them for 32 queries
  static constexpr int kThreads = 128 + 32 * kWarps;
  // staging: two buffers of 16 queries x (128 scores + 16 bytes) for each four warps
  static constexpr int kOutRow = 128 * 4 + 16;
  static constexpr int kOut = kStaged ? kWarps / 4 * 2 * 16 * kOutRow : 0;
};

template <int NT, int KB>
struct MxCfg : MxEpi<NT> {
  static constexpr int kAtoms = KB / 64, kSfB = 512 * kAtoms;   // scale tiles a stage and side
  static constexpr int kStage = kMxBM * KB + NT * KB + 2 * kSfB;
  static constexpr int kCtas = KB == 64 ? 4 : NT >= 64 ? 1 : 2;
  static constexpr int kBudget = (kCtas == 1 ? 226 : kCtas == 2 ? 112 : 55) * 1024 - 1024 - 512 -
                                 MxEpi<NT>::kOut;
  static constexpr int kStages = kBudget / kStage < kMxMaxStages ? kBudget / kStage : kMxMaxStages;
  static constexpr int kSmem = 1024 + kStages * kStage + MxEpi<NT>::kOut + 512;
  static constexpr int kCols = NT == 128 ? 512 : 4 * NT < 64 ? 64 : 4 * NT;  // TMEM columns
  static constexpr int kSfCol = 2 * NT;             // 32 columns of scales behind the sums
  static_assert(kStages >= 3 && kSfCol + 32 <= kCols && kCols * kCtas <= 512, "tile");
};

template <int NT, int KB>
struct MxPackCfg : MxEpi<NT> {
  static constexpr int kAtoms = KB / 64, kSfB = 512 * kAtoms;
  // vector tiles a step: with few queries a step's work is short against its barriers
  static constexpr int kSub = NT <= 32 && KB == 64 ? 2 : 1;
  static constexpr int kOne = kMxBM * KB + kSfB;    // a tile as it comes, and as the products read it
  static constexpr int kTile = kSub * kOne;
  static constexpr int kQ = NT * KB + kSfB;         // the queries' tile
  static constexpr int kMoveWarps = NT <= 32 ? 4 : 2;
  static constexpr int kThreads = MxEpi<NT>::kThreads + 32 * (kMoveWarps - 2);
  static constexpr int kCtas = NT == 128 || (NT == 64 && KB == 128) ? 1 : 2;
  static constexpr int kBufs = 2;                   // swizzled stages and accumulators
  static constexpr int kBudget = (kCtas == 1 ? 226 : 112) * 1024 - 1024 - 512 - MxEpi<NT>::kOut -
                                 kBufs * kTile - 2 * kQ;
  static constexpr int kRaw = kBudget / kTile < kMxMaxStages ? kBudget / kTile : kMxMaxStages;
  static constexpr int kSmem = 1024 + (kRaw + kBufs) * kTile + 2 * kQ + MxEpi<NT>::kOut + 512;
  // TMEM: the accumulators, the vectors' scales, the queries'
  static constexpr int kSfA = kBufs * kSub * NT, kSfQ = kSfA + kBufs * kSub * 4 * kAtoms;
  static constexpr int kNeed = kSfQ + 2 * 4 * kAtoms;
  static constexpr int kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  static_assert(kRaw >= 2 && kNeed <= 512 && kCols * kCtas <= 512, "tile");
};

struct MxBars {
  uint64_t full[kMxMaxStages], empty[kMxMaxStages];   // the ring
  uint64_t swz_full[2], swz_empty[2], q_full[2], q_empty[2];
  uint64_t s_full[2], s_empty[2], drain;              // accumulators
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(MxBars) <= 512, "barriers");

__device__ __forceinline__ void mx_timeout(int* status, MxBars* bars) {
  if (status) atomicCAS(status, FGMM_OK, FGMM_ERR_TIMEOUT);
  bars->abort = 1;
}

// The tiles of a CTA.  QFAST: queries fastest, so that a tile of long vectors is read from memory
// once; else vectors fastest, so that the queries' tile stays.
template <bool QFAST>
struct MxWalk {
  int64_t fast, slow, nfast, nslow, dfast, dslow;
  __device__ __forceinline__ MxWalk(int64_t vtiles, int64_t qtiles)
      : nfast(QFAST ? qtiles : vtiles), nslow(QFAST ? vtiles : qtiles) {
    fast = blockIdx.x % nfast, slow = blockIdx.x / nfast;
    dfast = gridDim.x % nfast, dslow = gridDim.x / nfast;
  }
  __device__ __forceinline__ bool more() const { return slow < nslow; }
  __device__ __forceinline__ void next() {
    fast += dfast, slow += dslow;
    if (fast >= nfast) fast -= nfast, ++slow;
  }
  __device__ __forceinline__ int64_t v() const { return QFAST ? slow : fast; }
  __device__ __forceinline__ int64_t q() const { return QFAST ? fast : slow; }
};

__device__ __forceinline__ void mx_cvt(float v, float& o) { o = v; }
__device__ __forceinline__ void mx_cvt(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// 16 staged queries leave as bulk copies: four a warp, eight lanes each.  One lane copies the aligned
// inside of a query's `len` scores, all write what lies before and behind it.  Element (query r,
// vector i) lies at st[r][phase_r + i], phase_r = (p0 + r dp) mod VN being what its address is off a
// 16-byte boundary; `out` is that of (query 0, vector 0).
template <typename T>
__device__ __forceinline__ void mx_rows_out(unsigned char* st, int row_bytes, int q, int lane, int rows,
                                            int len, int p0, int dp, T* out, int64_t ldo) {
  constexpr int VN = 16 / sizeof(T);
  const int r = 4 * q + (lane >> 3), ph = (p0 + r * dp) & (VN - 1), end = ph + len;
  const int a0 = (ph + VN - 1) & ~(VN - 1), a1 = end & ~(VN - 1);
  if (r < rows) {
    const T* from = reinterpret_cast<const T*>(st + r * row_bytes);
    T* to = out + r * ldo - ph;
    if ((lane & 7) == 0 && a1 > a0)
      ptx::bulk_store(to + a0, ptx::smem_u32(from + a0), (uint32_t)(a1 - a0) * sizeof(T));
    const int i = lane & 7;
    if (i >= ph && i < min(a0, end)) to[i] = from[i];
    if (max(a0, a1) + i < end) to[max(a0, a1) + i] = from[max(a0, a1) + i];
  }
  ptx::bulk_commit();
}

// The epilogue warps (`warp` from 0, a multiple of 4 in the CTA) of a CTA: scale, bias, rounding and
// the stores of every step of SUB vector tiles.
template <int NT, int SUB, int BUFS, bool QFAST, typename T>
__device__ __forceinline__ void mx_epilogue(int warp, MxBars* bars, unsigned char* outbuf, uint32_t tmem, int64_t n,
                                            int64_t m, int64_t vtiles, int64_t qtiles, float alpha,
                                            const float* __restrict__ bias, T* __restrict__ out,
                                            int64_t ldo, int* status) {
  using C = MxEpi<NT>;
  volatile int* abort = &bars->abort;
  const int lane = threadIdx.x & 31;
  constexpr int kColsWarp = NT * 4 / C::kWarps;          // columns a warp drains
  constexpr int kChunk = C::kStaged || kColsWarp < 32 ? 16 : 32;
  const int q = warp & 3, grp = warp >> 2, c0 = grp * kColsWarp;
  const uint32_t lane_base = (uint32_t)(q * 32) << 16;
  uint32_t buf = BUFS - 1, use = 1;                      // buffer and parity of its phase
  MxWalk<QFAST> ahead(vtiles, qtiles);
  float next_bias[SUB];
  auto load_bias = [&] {
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const int64_t row = (ahead.v() * SUB + u) * kMxBM + q * 32 + lane;
      next_bias[u] = bias && ahead.more() && row < n ? __ldg(bias + row) : 0.f;
    }
  };
  load_bias();
  for (MxWalk<QFAST> w(vtiles, qtiles); w.more(); w.next()) {
    const int64_t m0 = w.q() * NT + c0;
    if (++buf == BUFS) buf = 0, use ^= 1;
    float bvs[SUB];
#pragma unroll
    for (int u = 0; u < SUB; ++u) bvs[u] = next_bias[u];
    ahead.next();                                     // the next step's, while this one is drained
    load_bias();
    bool ok = ptx::mbar_wait_warp_soon(&bars->s_full[buf], use, abort);
    if (!ok) mx_timeout(status, bars);
    // the four warps of a group meet at barriers below: they go on or give up together
    if constexpr (C::kStaged) ok = ptx::named_all(1 + grp, 128, ok);
    if (!ok) break;
    ptx::tc_fence_after();
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) {
    const int64_t n0 = (w.v() * SUB + sub) * kMxBM, row = n0 + q * 32 + lane;
    const float bv = bvs[sub];
    const uint32_t acc = tmem + lane_base + (buf * SUB + sub) * NT + c0;
#pragma unroll
    for (int c = 0; c < kColsWarp; c += kChunk) {
      uint32_t u[kChunk];
      if constexpr (kChunk == 32) ptx::tmem_ld32(acc + c, u);
      else ptx::tmem_ld16(acc + c, u);
      ptx::tmem_wait_ld();
      if (sub + 1 == SUB && c + kChunk == kColsWarp) {  // all in registers: hand the accumulator back
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->s_empty[buf]);
      }
      const int64_t mc = m0 + c;
      const int rows = (int)min((int64_t)kChunk, m - mc);   // queries of the chunk (may be <= 0)
      if constexpr (C::kStaged) {
        constexpr int VN = 16 / sizeof(T);
        unsigned char* st = outbuf + (grp * 2 + ((c / kChunk) & 1)) * kChunk * C::kOutRow;
        // element (query r, vector i) of the chunk lies at st[r][phase_r + i], phase_r being what
        // its row's address is off a 16-byte boundary
        const int p0 = (int)(((uintptr_t)out / sizeof(T) + (uintptr_t)mc * ldo + n0) % VN);
        const int dp = (int)(ldo % VN);
        ptx::bulk_wait_read<1>();           // the buffer's last copies have read it
        ptx::named_sync(1 + grp, 128);
        T* mine = reinterpret_cast<T*>(st) + q * 32 + lane;
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
          mx_cvt(fmaf(alpha, __uint_as_float(u[e]), bv),
                 mine[e * (C::kOutRow / sizeof(T)) + ((p0 + e * dp) & (VN - 1))]);
        ptx::fence_proxy_async_smem();
        ptx::named_sync(1 + grp, 128);
        mx_rows_out<T>(st, C::kOutRow, q, lane, rows, (int)max((int64_t)0, min((int64_t)kMxBM, n - n0)), p0,
                       dp, out + mc * ldo + n0, ldo);
      } else if (row < n) {
        T* o = out + mc * ldo + row;
#pragma unroll
        for (int e = 0; e < kChunk; ++e, o += ldo)
          if (e < rows) mx_st(o, fmaf(alpha, __uint_as_float(u[e]), bv));
      }
    }
    }
  }
  if constexpr (C::kStaged) ptx::bulk_wait_read<0>();
}

template <int NT, int KB, typename T>
__global__ void __launch_bounds__(MxEpi<NT>::kThreads, MxCfg<NT, KB>::kCtas)
    mx4_scores_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmq,
                      const uint8_t* __restrict__ xs, const uint8_t* __restrict__ qs, int64_t n,
                      int64_t m, int nb, int64_t vtiles, int64_t qtiles, float alpha,
                      const float* __restrict__ bias, T* __restrict__ out, int64_t ldo, int* status) {
  using C = MxCfg<NT, KB>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* outbuf = ring + C::kStages * C::kStage;
  MxBars* bars = reinterpret_cast<MxBars*>(outbuf + C::kOut);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5;
  const int nkc = (nb + 3) / 4;                     // scale tiles (128 dimensions) of a row
  const int nst = (nkc + C::kAtoms - 1) / C::kAtoms;  // stages of a tile
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&bars->full[s], 1);
      ptx::mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&bars->s_full[b], 1);
      ptx::mbar_init(&bars->s_empty[b], C::kWarps);
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
  ptx::grid_wait();

  if (warp == 0) {
    {
      uint32_t it = 0, s = 0, ph = 1;               // ph: parity of the release to wait for
      bool ok = true;
      for (MxWalk<true> w(vtiles, qtiles); ok && w.more(); w.next()) {
        const uint8_t* xsf = xs + w.v() * nkc * 512;
        const uint8_t* qsf = qs + w.q() * nkc * 512;
        for (int k = 0; k < nst; ++k) {
          if (it >= C::kStages && !ptx::mbar_wait_all(&bars->empty[s], ph, abort)) {
            mx_timeout(status, bars);
            ok = false;
            break;
          }
          unsigned char* a = ring + s * C::kStage;
          unsigned char* b = a + kMxBM * KB;
          unsigned char* sf = b + NT * KB;
          const uint32_t sfb = min(nkc - C::kAtoms * k, C::kAtoms) * 512;
          if (ptx::elect_one()) {
            ptx::mbar_arrive_expect_tx(&bars->full[s], kMxBM * KB + NT * KB + 2 * sfb);
            ptx::tma_load_2d(a, &tmx, &bars->full[s], k * KB, (int)(w.v() * kMxBM));
            ptx::bulk_load(sf, xsf + k * C::kSfB, sfb, &bars->full[s]);
            ptx::tma_load_2d(b, &tmq, &bars->full[s], k * KB, (int)(w.q() * NT));
            ptx::bulk_load(sf + C::kSfB, qsf + k * C::kSfB, sfb, &bars->full[s]);
          }
          __syncwarp();
          ++it;
          if (++s == C::kStages) s = 0, ph ^= 1;
        }
      }
      if (!ok || *abort)  // let every copy this warp started land before the CTA exits
        for (uint32_t k = (it > C::kStages ? it - C::kStages : 0); k < it; ++k)
          ptx::mbar_drain(&bars->full[k % C::kStages], (k / C::kStages) & 1);
    }
  } else if (warp == 1) {
    {
      constexpr uint64_t kHiK = KB == 128 ? ptx::sw128_hi(16, 1024) : ptx::sw64_hi(16, 512);
      uint32_t s = 0, ph = 0, it = 0, j = 0;
      bool ok = true;
      for (MxWalk<true> w(vtiles, qtiles); ok && w.more(); w.next(), ++j) {
        const uint32_t buf = j & 1;
        if (j >= 2 && !ptx::mbar_wait_all(&bars->s_empty[buf], ((j >> 1) - 1) & 1, abort)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();  // the epilogue's reads of the buffer come before these products
        const uint32_t d_tmem = tmem + buf * NT;
        for (int k = 0; k < nst; ++k, ++it) {
          if (!ptx::mbar_wait_all(&bars->full[s], ph, abort)) {
            ok = false;
            break;
          }
          const uint32_t a = ptx::smem_u32(ring + s * C::kStage);
          const uint32_t b = a + kMxBM * KB, sf = b + NT * KB;
          const uint32_t sft = tmem + C::kSfCol + (it & 1) * 16;
          const int steps = min(2 * C::kAtoms, (nb + 1) / 2 - 2 * C::kAtoms * k);
          const uint64_t da = ptx::sw128_desc(a, kHiK), db = ptx::sw128_desc(b, kHiK);
          if (ptx::elect_one()) {
#pragma unroll
          for (int h = 0; h < C::kAtoms; ++h)
            if (2 * h < steps) {
              ptx::tmem_cp_32x128(sft + 4 * h, ptx::rows16_desc(sf + 512 * h));
              ptx::tmem_cp_32x128(sft + 8 + 4 * h, ptx::rows16_desc(sf + C::kSfB + 512 * h));
            }
#pragma unroll
          for (int q = 0; q < 2 * C::kAtoms; ++q)
            if (q < steps)
              ptx::mma_mxf4_ss(d_tmem, da + 2 * q, db + 2 * q, ptx::idesc_mxf4(kMxBM, NT, 2 * (q & 1)),
                               sft + 4 * (q >> 1), sft + 8 + 4 * (q >> 1), k > 0 || q > 0);
          ptx::mma_commit(&bars->empty[s]);
          }
          __syncwarp();
          if (++s == C::kStages) s = 0, ph ^= 1;
        }
        if (ok && ptx::elect_one()) ptx::mma_commit(&bars->s_full[buf]);
        __syncwarp();
      }
      if (!ok) {  // wait for the products already issued before TMEM is freed
        mx_timeout(status, bars);
        if (ptx::elect_one()) ptx::mma_commit(&bars->drain);
        ptx::mbar_drain(&bars->drain, 0);
      }
    }
  } else if (warp >= 4) {
    mx_epilogue<NT, 1, 2, true, T>(warp - 4, bars, outbuf, tmem, n, m, vtiles, qtiles, alpha, bias, out, ldo, status);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kCols);
  }
}

// Rows of at most KB bytes (nb <= KB / 16); vtiles counts steps of kSub vector tiles.
template <int NT, int KB, typename T>
__global__ void __launch_bounds__(MxPackCfg<NT, KB>::kThreads, MxPackCfg<NT, KB>::kCtas)
    mx4_scores_packed_kernel(const __grid_constant__ CUtensorMap tmq, const uint8_t* __restrict__ xc,
                             const uint8_t* __restrict__ xs, const uint8_t* __restrict__ qs, int64_t n,
                             int64_t m, int nb, int64_t vtiles, int64_t qtiles, float alpha,
                             const float* __restrict__ bias, T* __restrict__ out, int64_t ldo,
                             int* status) {
  using C = MxPackCfg<NT, KB>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* swz = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* qbuf = swz + C::kBufs * C::kTile;
  unsigned char* raw = qbuf + 2 * C::kQ;
  unsigned char* outbuf = raw + C::kRaw * C::kTile;
  MxBars* bars = reinterpret_cast<MxBars*>(outbuf + C::kOut);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nkc = (nb + 3) / 4;                     // scale tiles (128 dimensions) of a row
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kRaw; ++s) {
      ptx::mbar_init(&bars->full[s], 1);
      ptx::mbar_init(&bars->empty[s], C::kMoveWarps);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&bars->q_full[b], 1);
      ptx::mbar_init(&bars->q_empty[b], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      ptx::mbar_init(&bars->swz_full[b], C::kMoveWarps);
      ptx::mbar_init(&bars->swz_empty[b], 1);
      ptx::mbar_init(&bars->s_full[b], 1);
      ptx::mbar_init(&bars->s_empty[b], C::kWarps);
    }
    ptx::mbar_init(&bars->drain, 1);
    bars->abort = 0;
    ptx::fence_mbar_init();
  }
  // the part of a swizzled row behind its codes stays 0 (and so do rows behind the last vector,
  // until codes of an earlier tile lie there, whose scores are not written)
  for (int i = threadIdx.x; i < C::kBufs * C::kTile / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(swz)[i] = make_uint4(0u, 0u, 0u, 0u);
  ptx::fence_proxy_async_smem();
  if (warp == 1) {
    ptx::tmem_alloc(&bars->tmem, C::kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem;
  ptx::grid_wait();

  if (warp == 0) {
    {
      uint32_t it = 0, s = 0, ph = 1, jq = 0;       // ph: parity of the release to wait for
      int64_t qt = -1;
      bool ok = true;
      for (MxWalk<false> w(vtiles, qtiles); ok && w.more(); w.next()) {
        if (w.q() != qt) {                          // the next tile of queries
          qt = w.q();
          const uint32_t b = jq & 1;
          if (jq >= 2 && !ptx::mbar_wait_all(&bars->q_empty[b], ((jq >> 1) - 1) & 1, abort)) ok = false;
          if (!ok) break;
          if (ptx::elect_one()) {
            ptx::mbar_arrive_expect_tx(&bars->q_full[b], NT * KB + nkc * 512);
            ptx::tma_load_2d(qbuf + b * C::kQ, &tmq, &bars->q_full[b], 0, (int)(qt * NT));
            ptx::bulk_load(qbuf + b * C::kQ + NT * KB, qs + qt * nkc * 512, nkc * 512, &bars->q_full[b]);
          }
          __syncwarp();
          ++jq;
        }
        if (it >= C::kRaw && !ptx::mbar_wait_all(&bars->empty[s], ph, abort)) {
          ok = false;
          break;
        }
        const int64_t v0 = w.v() * C::kSub * kMxBM;
        const int rows = (int)min((int64_t)C::kSub * kMxBM, n - v0);
        const uint32_t bytes = (uint32_t)rows * nb * 16, sfb = (rows + 127) / 128 * nkc * 512;
        unsigned char* to = raw + s * C::kTile;
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(&bars->full[s], bytes + sfb);
          ptx::bulk_load(to, xc + v0 * nb * 16, bytes, &bars->full[s]);
          ptx::bulk_load(to + C::kSub * kMxBM * KB, xs + v0 / kMxBM * nkc * 512, sfb, &bars->full[s]);
        }
        __syncwarp();
        ++it;
        if (++s == C::kRaw) s = 0, ph ^= 1;
      }
      if (!ok) mx_timeout(status, bars);
      if (!ok || *abort) {  // let every copy this warp started land before the CTA exits
        for (uint32_t k = (it > C::kRaw ? it - C::kRaw : 0); k < it; ++k)
          ptx::mbar_drain(&bars->full[k % C::kRaw], (k / C::kRaw) & 1);
        for (uint32_t k = (jq > 2 ? jq - 2 : 0); k < jq; ++k)
          ptx::mbar_drain(&bars->q_full[k & 1], (k >> 1) & 1);
      }
    }
  } else if (warp == 1) {
    {
      constexpr uint64_t kHiK = KB == 128 ? ptx::sw128_hi(16, 1024) : ptx::sw64_hi(16, 512);
      const int steps = (nb + 1) / 2;
      uint32_t j = 0, jq = 0, buf = C::kBufs - 1, use = 1;   // buffer and parity of its phase
      int64_t qt = -1;
      bool ok = true;
      for (MxWalk<false> w(vtiles, qtiles); ok && w.more(); ++j) {
        if (++buf == C::kBufs) buf = 0, use ^= 1;
        // (the scale columns of the buffer's last step are free with its sums)
        if (j >= C::kBufs && !ptx::mbar_wait_all(&bars->s_empty[buf], use ^ 1, abort)) ok = false;
        if (!ok) break;
        ptx::tc_fence_after();  // the epilogue's reads of the buffer come before these products
        if (w.q() != qt) {
          qt = w.q();
          ok = ptx::mbar_wait_all(&bars->q_full[jq & 1], (jq >> 1) & 1, abort);
          if (!ok) break;
          const uint32_t sf = ptx::smem_u32(qbuf + (jq & 1) * C::kQ + NT * KB);
          if (ptx::elect_one())
            for (int h = 0; h < nkc; ++h)
              ptx::tmem_cp_32x128(tmem + C::kSfQ + (jq & 1) * 4 * C::kAtoms + 4 * h,
                                  ptx::rows16_desc(sf + 512 * h));
          __syncwarp();
          ++jq;
        }
        const uint32_t sfq = tmem + C::kSfQ + ((jq - 1) & 1) * 4 * C::kAtoms;
        ok = ptx::mbar_wait_all(&bars->swz_full[buf], use, abort);
        if (!ok) break;
        const uint64_t db = ptx::sw128_desc(ptx::smem_u32(qbuf + ((jq - 1) & 1) * C::kQ), kHiK);
        if (ptx::elect_one()) {
#pragma unroll
        for (int u = 0; u < C::kSub; ++u) {
          const uint32_t a = ptx::smem_u32(swz + buf * C::kTile + u * C::kOne), sf = a + kMxBM * KB;
          const uint32_t sfa = tmem + C::kSfA + (buf * C::kSub + u) * 4 * C::kAtoms;
          for (int h = 0; h < nkc; ++h)
            ptx::tmem_cp_32x128(sfa + 4 * h, ptx::rows16_desc(sf + 512 * h));
          const uint64_t da = ptx::sw128_desc(a, kHiK);
#pragma unroll
          for (int q = 0; q < 2 * C::kAtoms; ++q)
            if (q < steps)
              ptx::mma_mxf4_ss(tmem + (buf * C::kSub + u) * NT, da + 2 * q, db + 2 * q,
                               ptx::idesc_mxf4(kMxBM, NT, 2 * (q & 1)), sfa + 4 * (q >> 1),
                               sfq + 4 * (q >> 1), q > 0);
        }
        ptx::mma_commit(&bars->swz_empty[buf]);
        ptx::mma_commit(&bars->s_full[buf]);
        }
        __syncwarp();
        w.next();
        if (w.more() && w.q() != qt && ptx::elect_one()) ptx::mma_commit(&bars->q_empty[(jq - 1) & 1]);
        __syncwarp();
      }
      if (!ok) {  // wait for the products already issued before TMEM is freed
        mx_timeout(status, bars);
        if (ptx::elect_one()) ptx::mma_commit(&bars->drain);
        ptx::mbar_drain(&bars->drain, 0);
      }
    }
  } else if (warp < 4 || warp >= 4 + C::kWarps) {
    // from the order of memory to the swizzled one: 16-byte chunk c of row r goes to chunk
    // c ^ (r mod 8) of 128-byte rows, c ^ (r / 2 mod 4) of 64-byte rows
    const int t = threadIdx.x - 64 - (warp < 4 ? 0 : 32 * C::kWarps);
    constexpr int kMove = 32 * C::kMoveWarps;
    const uint32_t inv = (65536u + nb - 1) / nb;     // i / nb for i < 2048
    uint32_t s = 0, ph = 0, j = 0, buf = C::kBufs - 1, use = 1;
    for (MxWalk<false> w(vtiles, qtiles); w.more(); w.next(), ++j) {
      if (++buf == C::kBufs) buf = 0, use ^= 1;
      bool ok = ptx::mbar_wait_warp_soon(&bars->full[s], ph, abort);
      if (ok && j >= C::kBufs) ok = ptx::mbar_wait_warp_soon(&bars->swz_empty[buf], use ^ 1, abort);
      if (!ok) {
        mx_timeout(status, bars);
        break;
      }
      const uint4* from = reinterpret_cast<const uint4*>(raw + s * C::kTile);
      uint4* to = reinterpret_cast<uint4*>(swz + buf * C::kTile);
      const int rows = (int)min((int64_t)C::kSub * kMxBM, n - w.v() * C::kSub * kMxBM);
#pragma unroll 4
      for (int i = t; i < rows * nb; i += kMove) {
        const uint32_t r = (uint32_t)i * inv >> 16, c = i - r * nb;
        to[(r >> 7) * (C::kOne / 16) + (r & 127) * (KB / 16) + (c ^ (KB == 128 ? r & 7 : r >> 1 & 3))] =
            from[i];
      }
      for (int i = t; i < nkc * 32; i += kMove)
#pragma unroll
        for (int u = 0; u < C::kSub; ++u)
          if (128 * u < rows)
            to[u * (C::kOne / 16) + kMxBM * KB / 16 + i] =
                from[C::kSub * kMxBM * KB / 16 + u * nkc * 32 + i];
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&bars->swz_full[buf]);
        ptx::mbar_arrive(&bars->empty[s]);
      }
      if (++s == C::kRaw) s = 0, ph ^= 1;
    }
  } else {
    mx_epilogue<NT, C::kSub, C::kBufs, false, T>(warp - 4, bars, outbuf, tmem, n, m, vtiles, qtiles, alpha, bias, out, ldo, status);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kCols);
  }
}

// ------------------------------------------------------------------ scores by pairs of CTAs
// Many queries of long vectors: the products decide, and what bounds them is how fast operands come
// into shared memory (TMA moves about 30 bytes a clock and SM).  A pair of CTAs shares a tile of 256
// vectors x 256 queries: each loads its 128 vectors and half of the queries, 32 KB for 128 x 256 x 256
// products, half of what a tile of 128 x 128 needs.  The first CTA issues the products of both, and the
// copies of both are counted on its barriers (a thread of the second passing on that its stage is full
// cost a third of the time).
//
// Two accumulators of 256 columns and the scales do not fit into 512 columns, so the accumulators
// overlap by 32: the epilogue drains those first, and the next tile's products wait for them alone.
template <typename T>
struct MxPairCfg {
  static constexpr int NT = 256, KB = 128;
  static constexpr int kA = kMxBM * KB, kB = NT / 2 * KB, kSf = 1024;
  static constexpr int kStage = kA + kB + 3 * kSf;  // own vectors, half of the queries; scales: own, all
  static constexpr int kGroups = 4, kWarps = 4 * kGroups, kThreads = 128 + 32 * kWarps;
  static constexpr int kOutRow = 128 * sizeof(T) + 16;
  static constexpr int kOut = kGroups * 2 * 16 * kOutRow;
  static constexpr int kBudget = 226 * 1024 - 1024 - 512 - kOut;
  static constexpr int kStages = kBudget / kStage < kMxMaxStages ? kBudget / kStage : kMxMaxStages;
  static constexpr int kSmem = 1024 + kStages * kStage + kOut + 512;
  static constexpr int kOverlap = 32, kAcc1 = NT - kOverlap, kSfCol = 2 * NT - kOverlap;
  static_assert(kStages >= 3 && kSfCol + 2 * 12 <= 512, "tile");
};

struct MxPairBars {
  uint64_t full[kMxMaxStages], empty[kMxMaxStages];
  uint64_t s_full[2], s_empty[2], overlap, drain;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(MxPairBars) <= 512, "barriers");

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MxPairCfg<T>::kThreads, 1)
    mx4_scores_pair_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmq,
                           const __grid_constant__ CUtensorMap tmxs, const __grid_constant__ CUtensorMap tmqs,
                           int64_t n, int64_t m, int nb, int64_t vpairs, int64_t qtiles, float alpha,
                           const float* __restrict__ bias, T* __restrict__ out, int64_t ldo, int* status) {
  using C = MxPairCfg<T>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* outbuf = ring + C::kStages * C::kStage;
  MxPairBars* bars = reinterpret_cast<MxPairBars*>(outbuf + C::kOut);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1;
  const int nkc = (nb + 3) / 4, nst = (nkc + 1) / 2;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(&bars->full[s], 1);
      ptx::mbar_init(&bars->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&bars->s_full[b], 1);
      ptx::mbar_init(&bars->s_empty[b], 2 * C::kWarps);
    }
    ptx::mbar_init(&bars->overlap, 2 * 4);
    ptx::mbar_init(&bars->drain, 1);
    bars->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&bars->tmem, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem;
  ptx::grid_wait();
  auto timeout = [&] {
    if (status) atomicCAS(status, FGMM_OK, FGMM_ERR_TIMEOUT);
    bars->abort = 1;
  };
  // tiles of the pair, queries fastest
  const int64_t p0 = blockIdx.x >> 1, np = gridDim.x >> 1, ntiles = vpairs * qtiles;

  if (warp == 0) {
    {
      uint32_t it = 0, s = 0, ph = 1;
      bool ok = true;
      for (int64_t t = p0; ok && t < ntiles; t += np) {
        const int64_t vp = t / qtiles, qt = t - vp * qtiles;
        const int vt = (int)(2 * vp + rank), qh = (int)(qt * C::NT + rank * (C::NT / 2));
        for (int k = 0; k < nst; ++k) {             // (what is behind the last row or block reads as 0)
          if (it >= C::kStages && !ptx::mbar_wait_all(&bars->empty[s], ph, abort)) {
            timeout();
            ok = false;
            break;
          }
          unsigned char* a = ring + s * C::kStage;
          unsigned char* sf = a + C::kA + C::kB;
          const uint32_t bar = ptx::cluster_addr(&bars->full[s], 0);
          if (ptx::elect_one()) {
            if (rank == 0) ptx::mbar_arrive_expect_tx(&bars->full[s], 2 * C::kStage);
            ptx::tma_load_2d_pair(a, &tmx, bar, k * C::KB, vt * kMxBM);
            ptx::tma_load_2d_pair(a + C::kA, &tmq, bar, k * C::KB, qh);
            ptx::tma_load_3d_pair(sf, &tmxs, bar, 0, 2 * k, vt);
            ptx::tma_load_3d_pair(sf + C::kSf, &tmqs, bar, 0, 2 * k, (int)(2 * qt));
          }
          __syncwarp();
          ++it;
          if (++s == C::kStages) s = 0, ph ^= 1;
        }
      }
      if (!ok || *abort) {  // let every copy this warp started land before the CTA exits
        if (rank == 0)
          for (uint32_t k = (it > C::kStages ? it - C::kStages : 0); k < it; ++k)
            ptx::mbar_drain(&bars->full[k % C::kStages], (k / C::kStages) & 1);
        else                                        // (its copies are counted over there: 1 ms is ample)
          for (const uint64_t t0 = ptx::globaltimer_ns(); ptx::globaltimer_ns() - t0 < 1000000;) {}
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint64_t kHiK = ptx::sw128_hi(16, 1024);
      uint32_t s = 0, ph = 0, j = 0, cp = 0;
      bool ok = true;
      for (int64_t t = p0; ok && t < ntiles; t += np, ++j) {
        const uint32_t buf = j & 1;
        if (j >= 2) ok = ptx::mbar_wait_cluster_all(&bars->s_empty[buf], ((j >> 1) - 1) & 1, abort);
        if (ok && j >= 1) ok = ptx::mbar_wait_cluster_all(&bars->overlap, (j - 1) & 1, abort);
        if (!ok) break;
        ptx::tc_fence_after();  // both epilogues' reads of these columns come before the products
        const uint32_t d_tmem = tmem + (buf ? C::kAcc1 : 0);
        for (int k = 0; k < nst; ++k) {
          ok = ptx::mbar_wait_cluster_all(&bars->full[s], ph, abort);
          if (!ok) break;
          const uint32_t a = ptx::smem_u32(ring + s * C::kStage), sf = a + C::kA + C::kB;
          const uint64_t da = ptx::sw128_desc(a, kHiK), db = ptx::sw128_desc(a + C::kA, kHiK);
          const int steps = min(4, (nb + 1) / 2 - 4 * k);
          if (ptx::elect_one()) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (2 * h < steps) {
              // 12 columns of scales for 128 dimensions: the vectors' 4, the queries' 8
              const uint32_t sft = tmem + C::kSfCol + ((cp + h) & 1) * 12;
              ptx::tmem_cp_32x128_pair(sft, ptx::rows16_desc(sf + 512 * h));
              ptx::tmem_cp_32x128_pair(sft + 4, ptx::rows16_desc(sf + C::kSf + 512 * h));
              ptx::tmem_cp_32x128_pair(sft + 8, ptx::rows16_desc(sf + 2 * C::kSf + 512 * h));
#pragma unroll
              for (int q = 2 * h; q < 2 * h + 2; ++q)
                if (q < steps)
                  ptx::mma_mxf4_pair(d_tmem, da + 2 * q, db + 2 * q, ptx::idesc_mxf4(256, C::NT, 2 * (q & 1)),
                                     sft, sft + 4, k > 0 || q > 0);
            }
          ptx::mma_commit_pair(&bars->empty[s]);
          }
          __syncwarp();
          cp += (steps + 1) / 2;
          if (++s == C::kStages) s = 0, ph ^= 1;
        }
        if (ok && ptx::elect_one()) ptx::mma_commit_pair(&bars->s_full[buf]);
        __syncwarp();
      }
      if (!ok) {  // wait for the products already issued before TMEM is freed
        timeout();
        if (ptx::elect_one()) ptx::mma_commit_pair(&bars->drain);
        ptx::mbar_drain(&bars->drain, 0);
      }
    }
  } else if (warp >= 4) {
    constexpr int VN = 16 / sizeof(T);
    const int q = warp & 3, grp = (warp - 4) >> 2;
    uint32_t j = 0;
    auto bias_of = [&](int64_t t) {
      const int64_t row = (2 * (t / qtiles) + rank) * kMxBM + q * 32 + lane;
      return bias && t < ntiles && row < n ? __ldg(bias + row) : 0.f;
    };
    float next_bias = bias_of(p0);
    for (int64_t t = p0; t < ntiles; t += np, ++j) {
      const int64_t vp = t / qtiles, qt = t - vp * qtiles;
      const uint32_t buf = j & 1;
      const int64_t n0 = (2 * vp + rank) * kMxBM;
      const float bv = next_bias;
      next_bias = bias_of(t + np);                  // the next tile's, while this one is drained
      bool ok = ptx::mbar_wait_warp_soon(&bars->s_full[buf], (j >> 1) & 1, abort);
      if (!ok) timeout();
      ok = ptx::named_all(1 + grp, 128, ok);        // the four warps of a group go on or give up together
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (buf ? C::kAcc1 : 0) + grp * 64;
      const int len = (int)max((int64_t)0, min((int64_t)kMxBM, n - n0));
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {                 // 32 columns at a time, the shared ones first
        const int c = 32 * (buf ? i : 1 - i);
        uint32_t u[32];
        ptx::tmem_ld32(acc + c, u);
        ptx::tmem_wait_ld();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (i == 0 && grp == (buf ? 0 : C::kGroups - 1)) ptx::mbar_arrive_cluster(&bars->overlap, 0);
          if (i == 1) ptx::mbar_arrive_cluster(&bars->s_empty[buf], 0);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int64_t mc = qt * C::NT + grp * 64 + c + 16 * half;
          const int rows = (int)min((int64_t)16, m - mc);
          unsigned char* st = outbuf + (grp * 2 + half) * 16 * C::kOutRow;
          const int pm = (int)(((uintptr_t)out / sizeof(T) + (uintptr_t)mc * ldo + n0) % VN);
          const int dp = (int)(ldo % VN);
          ptx::bulk_wait_read<1>();
          ptx::named_sync(1 + grp, 128);
          T* mine = reinterpret_cast<T*>(st) + q * 32 + lane;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            mx_cvt(fmaf(alpha, __uint_as_float(u[16 * half + e]), bv),
                   mine[e * (C::kOutRow / sizeof(T)) + ((pm + e * dp) & (VN - 1))]);
          ptx::fence_proxy_async_smem();
          ptx::named_sync(1 + grp, 128);
          mx_rows_out<T>(st, C::kOutRow, q, lane, rows, len, pm, dp, out + mc * ldo + n0, ldo);
        }
      }
    }
    ptx::bulk_wait_read<0>();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();                              // the other CTA's products read this one's memory
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// Rows of codes as boxes of `box_bytes` (64 or 128, swizzled as wide) x `box_rows`; what lies beyond
// a row or the last row is 0.
bool mx_tmap(CUtensorMap* map, const uint8_t* codes, int nb, int64_t rows, int box_bytes,
             int box_rows) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)nb * 16, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)nb * 16};
  const cuuint32_t box[2] = {(cuuint32_t)box_bytes, (cuuint32_t)box_rows};
  const cuuint32_t one[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles [rows of tiles][tiles of a row][512 bytes] as boxes of 2 of a row x `box_rows`.
bool mx_tmap_scales(CUtensorMap* map, const uint8_t* scales, int nb, int64_t rows, int box_rows) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t nkc = (cuuint64_t)(nb + 3) / 4;
  const cuuint64_t dims[3] = {128, nkc, (cuuint64_t)(rows + 127) / 128};
  const cuuint64_t strides[2] = {512, 512 * nkc};
  const cuuint32_t box[3] = {128, 2, (cuuint32_t)box_rows}, one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(scales), dims, strides, box,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
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

// Launch that may begin before the encoding of its operands has ended (grid_wait in the kernels).
template <typename... P, typename... A>
cudaError_t mx_launch(void (*kernel)(P...), unsigned grid, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Grid and attributes of a kernel with configuration C; its query and vector tiles.
template <typename C, typename K>
cudaError_t mx_grid_of(K* kernel, int64_t tiles, unsigned* grid) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t slots = (int64_t)sms * C::kCtas;
  *grid = (unsigned)(tiles < slots ? tiles : slots);
  return e;
}

template <int NT, int KB, typename T>
cudaError_t mx_scores(const MxArgs& a) {
  const int64_t qt = (a.m + NT - 1) / NT, vt = (a.n + kMxBM - 1) / kMxBM;
  unsigned grid = 0;
  CUtensorMap tmx, tmq;
  cudaError_t e;
  if (!mx_tmap(&tmq, a.qc, a.nb, a.m, KB, NT)) return cudaErrorInvalidValue;
  // Bulk copies for rows shorter than a box.  Rows that fill one come by boxes where that is faster: at
  // 256 dimensions up to 64 queries (10^6 vectors, boxes and copies: one query 29.0 and 34.8 us, 16
  // 35.6 and 35.9; 64 and 500000: 41.3 and 45.0; 1000 x 100003 fp32: 90.9 and 83.7), at 128 for one
  // query (15.9 and 21.4 us; two queries 25.6 and 21.6).
  constexpr bool kBoxes = KB == 128 || NT == 16;
  const bool full = 16 * a.nb == KB && a.m <= (KB == 128 ? 64 : 1);
  if (!kBoxes || (16 * a.nb <= KB && !full)) {
    using C = MxPackCfg<NT, KB>;
    const int64_t steps = (vt + C::kSub - 1) / C::kSub;
    auto* k = mx4_scores_packed_kernel<NT, KB, T>;
    if ((e = mx_grid_of<C>(k, steps * qt, &grid)) != cudaSuccess) return e;
    return mx_launch(k, grid, C::kThreads, C::kSmem, a.s, tmq, a.xc, a.xs, a.qs, a.n, a.m, a.nb, steps, qt,
                     a.alpha, a.bias, static_cast<T*>(a.out), a.ldo, a.status);
  }
  if constexpr (kBoxes) {
    using C = MxCfg<NT, KB>;
    auto* k = mx4_scores_kernel<NT, KB, T>;
    if ((e = mx_grid_of<C>(k, vt * qt, &grid)) != cudaSuccess) return e;
    if (!mx_tmap(&tmx, a.xc, a.nb, a.n, KB, kMxBM)) return cudaErrorInvalidValue;
    e = mx_launch(k, grid, C::kThreads, C::kSmem, a.s, tmx, tmq, a.xs, a.qs, a.n, a.m, a.nb, vt, qt, a.alpha,
                  a.bias, static_cast<T*>(a.out), a.ldo, a.status);
  }
  return e;
}

template <typename T>
cudaError_t mx_scores_pair(const MxArgs& a) {
  using C = MxPairCfg<T>;
  CUtensorMap tmx, tmq, tmxs, tmqs;
  if (!mx_tmap(&tmx, a.xc, a.nb, a.n, C::KB, kMxBM) || !mx_tmap(&tmq, a.qc, a.nb, a.m, C::KB, C::NT / 2) ||
      !mx_tmap_scales(&tmxs, a.xs, a.nb, a.n, 1) || !mx_tmap_scales(&tmqs, a.qs, a.nb, a.m, 2))
    return cudaErrorInvalidValue;
  auto* k = mx4_scores_pair_kernel<T>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  int dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t vp = (a.n + 2 * kMxBM - 1) / (2 * kMxBM), qt = (a.m + C::NT - 1) / C::NT;
  const int64_t pairs = vp * qt < sms / 2 ? vp * qt : sms / 2;
  return mx_launch(k, (unsigned)(2 * pairs), C::kThreads, C::kSmem, a.s, tmx, tmq, tmxs, tmqs, a.n, a.m, a.nb,
                   vp, qt, a.alpha, a.bias, static_cast<T*>(a.out), a.ldo, a.status);
}

template <int KB, typename T>
cudaError_t mx_scores_nt(const MxArgs& a) {
  if (KB == 128 && a.nb > 8 && a.m > 128 && a.n > 128) return mx_scores_pair<T>(a);
  if (a.m <= 16) return mx_scores<16, KB, T>(a);
  if (a.m <= 32) return mx_scores<32, KB, T>(a);
  if (a.m <= 64) return mx_scores<64, KB, T>(a);
  return mx_scores<128, KB, T>(a);
}
template <typename T>
cudaError_t mx_scores_kb(const MxArgs& a) {
  return a.nb <= 4 ? mx_scores_nt<64, T>(a) : mx_scores_nt<128, T>(a);
}

template <typename T>
cudaError_t mx_encode(const T* X, int64_t n, int D, int64_t ldx, int nb, int nkc, uint8_t* codes,
                      uint8_t* scales, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const auto rows_at = [&](int b) { return (uintptr_t)X % b == 0 && ldx * sizeof(T) % b == 0; };
  const int pad = 4 * nkc - nb;
  const bool tiles = pad <= nkc / 2 && rows_at(16);   // at most an eighth of the lanes idle
  // fill the device, fewer blocks when there is less.  On the padded walk two pieces a thread at every
  // size, against one: fp32 x 128, 5000 rows 2.70 and 2.77 us, 20000 3.9 and 4.9, 100000 11.2 and 14.3;
  // bf16 x 960, 2000 rows 2.9 and 3.7, 20000 11.3 and 17.7 (the grid ends at 32 blocks an SM either way).
  int64_t blocks = (n + 127) / 128 * 128 * (tiles ? 4 * nkc : nb) * sizeof(T);
  blocks = (blocks + kMxThreads - 1) / kMxThreads;
  if (tiles) blocks = (blocks + 1) / 2;
  const int64_t most = (int64_t)sms * (tiles ? 32 : 16);
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  auto* k = tiles ? (rows_at(32) ? mx4_encode_kernel<T, 32, true> : mx4_encode_kernel<T, 16, true>)
            : rows_at(16) ? mx4_encode_kernel<T, 16, false>
            : rows_at(8)  ? mx4_encode_kernel<T, 8, false>
            : rows_at(4)  ? mx4_encode_kernel<T, 4, false>
                          : mx4_encode_kernel<T, (int)sizeof(T), false>;
  k<<<grid, kMxThreads, 0, s>>>(X, n, D, ldx, nb, nkc, codes, scales);
  return cudaGetLastError();
}

template <typename T, int BYTES, int AT>
cudaError_t mx_decode_by(const uint8_t* codes, const uint8_t* scales, int64_t n, int D, T* out,
                         int64_t ldo, cudaStream_t s) {
  constexpr int N = BYTES / sizeof(T);
  const int nb = (D + 31) / 32, nkc = (nb + 3) / 4, segs = (D + N - 1) / N;
  const int64_t pieces = (n + 127) / 128 * 32 * segs, blocks = (pieces + kMxThreads - 1) / kMxThreads;
  return mx_launch(mx4_decode_kernel<T, BYTES, AT>, (unsigned)(blocks < (1 << 30) ? blocks : (1 << 30)),
                   kMxThreads, 0, s, codes, scales, n, D, nb, nkc, segs, pieces, out, ldo);
}
template <typename T>
cudaError_t mx_decode(const uint8_t* codes, const uint8_t* scales, int64_t n, int D, T* out, int64_t ldo,
                      cudaStream_t s) {
  const auto rows_at = [&](int b) { return (uintptr_t)out % b == 0 && ldo * sizeof(T) % b == 0; };
  if (rows_at(32)) return mx_decode_by<T, 32, 32>(codes, scales, n, D, out, ldo, s);
  if (rows_at(16)) return mx_decode_by<T, 16, 16>(codes, scales, n, D, out, ldo, s);
  if (rows_at(8)) return mx_decode_by<T, 16, 8>(codes, scales, n, D, out, ldo, s);
  if constexpr (sizeof(T) == 2) {
    if (!rows_at(4)) return mx_decode_by<T, 8, 2>(codes, scales, n, D, out, ldo, s);
  }
  return mx_decode_by<T, 16, 4>(codes, scales, n, D, out, ldo, s);
}

}  // namespace

// ------------------------------------------------------------------ launchers
cudaError_t launch_mx4_encode(const void* X, int x_dtype, int64_t n, int D, int64_t ldx,
                              uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  const int nb = (D + 31) / 32, nkc = (nb + 3) / 4;
  if (x_dtype == FGMM_F32)
    return mx_encode(static_cast<const float*>(X), n, D, ldx, nb, nkc, codes, scales, s);
  return mx_encode(static_cast<const __nv_bfloat16*>(X), n, D, ldx, nb, nkc, codes, scales, s);
}

cudaError_t launch_mx4_decode(const uint8_t* codes, const uint8_t* scales, int64_t n, int D,
                              void* out, int out_dtype, int64_t ldo, cudaStream_t s) {
  if (out_dtype == FGMM_F32) return mx_decode(codes, scales, n, D, static_cast<float*>(out), ldo, s);
  return mx_decode(codes, scales, n, D, static_cast<__nv_bfloat16*>(out), ldo, s);
}

cudaError_t launch_mx4_scores(const uint8_t* q_codes, const uint8_t* q_scales, int64_t m,
                              const uint8_t* codes, const uint8_t* scales, int64_t n, int D,
                              float alpha, const float* bias, void* out, int out_dtype,
                              int64_t ldo, int* status, cudaStream_t s) {
  const MxArgs a = {q_codes, q_scales, codes, scales, m, n, (D + 31) / 32, alpha, bias, out, ldo,
                    status, s};
  return out_dtype == FGMM_F32 ? mx_scores_kb<float>(a) : mx_scores_kb<__nv_bfloat16>(a);
}

cudaError_t mx4_status_word(int** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), mx_status_word);
}

}  // namespace fgmm
