// f8_quant.cu -- block-scaled E4M3 quantisation.
//
// For a block with largest magnitude a (at least kTinyAmax): scale s = a / 448
// and q = 448 x / a rounded to the nearest E4M3 value, ties to even; an entry
// stands for q * s.  A block is 128 consecutive entries of a row (rows), of a
// column (columns: the result is stored transposed, so that its 128 entries
// are contiguous too), or a 128 x 128 tile.
//
// The quotient is rounded to fp32 correctly before it is rounded to E4M3, as
// an IEEE division would: q0 = n r, q1 = q0 + r (n - q0 d) with r = 1/d
// correctly rounded (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990), here n = 0.875 x and d = a / 512, so
// that neither side overflows and n is exact for 16-bit entries.  Three
// operations per entry instead of a division's ten keep the pass bound by
// memory.  An entry that is inf or NaN makes its block's scale inf or NaN,
// and every value of the block then stands for NaN.
//
// 8192 x 4096 bf16: rows 19.3 us, columns 20.0, tiles 19.0 (the bytes at the copy
// rate: 15.2), both 28.3 (20.4); fp32 31, 33, 31 (25) and 41 (30).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <climits>
#include <cstdint>
#include <cstring>

#include "f8_act.cuh"
#include "f8_kernels.h"

namespace rg {
namespace {

constexpr uint32_t kTinyBits = 0x21800000u;  // 2^-60
constexpr int kTile = 128;

// Eight entries of a row as loaded, and largest magnitudes of them ("mags"): of
// 16-bit entries two to a word, compared by the packed maximum that keeps a
// NaN; of fp32 entries one to a word, compared as bit patterns, where NaN lies
// above inf.
template <typename T>
struct Entries {
  static constexpr int kWords = 4;
  static constexpr int kPer = 2;  // entries per word
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  }
  __device__ __forceinline__ void load_words(const T* p) {  // from a 4-byte boundary
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
  }
  __device__ __forceinline__ void set(int i, T v) {
    uint16_t h;
    memcpy(&h, &v, 2);
    w[i >> 1] |= (uint32_t)h << (16 * (i & 1));
  }
  static __device__ __forceinline__ uint32_t mag(uint32_t a) { return a & 0x7FFF7FFFu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b);
  static __device__ __forceinline__ float lo(uint32_t a);
  static __device__ __forceinline__ float hi(uint32_t a);
  __device__ __forceinline__ float at(int i) const { return i & 1 ? hi(w[i >> 1]) : lo(w[i >> 1]); }
  // the larger of a mag's two entries, as an fp32 bit pattern
  static __device__ __forceinline__ uint32_t top(uint32_t m) {
    return max(__float_as_uint(lo(m)), __float_as_uint(hi(m)));
  }
};
template <>
__device__ __forceinline__ uint32_t Entries<__nv_bfloat16>::larger(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <>
__device__ __forceinline__ float Entries<__nv_bfloat16>::lo(uint32_t a) { return __uint_as_float(a << 16); }
template <>
__device__ __forceinline__ float Entries<__nv_bfloat16>::hi(uint32_t a) { return __uint_as_float(a & 0xFFFF0000u); }
template <>
__device__ __forceinline__ uint32_t Entries<__half>::larger(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <>
__device__ __forceinline__ float Entries<__half>::lo(uint32_t a) {
  return __half2float(__ushort_as_half((unsigned short)a));
}
template <>
__device__ __forceinline__ float Entries<__half>::hi(uint32_t a) {
  return __half2float(__ushort_as_half((unsigned short)(a >> 16)));
}
template <>
struct Entries<float> {
  static constexpr int kWords = 8;
  static constexpr int kPer = 1;
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* p) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p)), v = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
  }
  __device__ __forceinline__ void load_words(const float* p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
  }
  __device__ __forceinline__ void set(int i, float v) { w[i] = __float_as_uint(v); }
  static __device__ __forceinline__ uint32_t mag(uint32_t a) { return a & 0x7FFFFFFFu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
  static __device__ __forceinline__ uint32_t top(uint32_t m) { return m; }
};

// Eight entries from p, of which `left` exist; missing ones read as 0.  unit: all rows
// start on boundaries of so many bytes.  (8192 rows of bf16: 4096 columns 17.7 us, 4094
// 24.4, entry by entry 34; of 4095 columns 35, shifted out of the words around them no less.)
template <typename T>
__device__ __forceinline__ void load8(Entries<T>& e, const T* p, long long left, int unit) {
  if (unit == 16 && left >= 8) {
    e.load(p);
  } else if (unit >= 4 && left >= 8) {
    e.load_words(p);
  } else {
#pragma unroll
    for (int i = 0; i < Entries<T>::kWords; ++i) e.w[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) e.set(i, p[i]);
  }
}
template <typename T>
__device__ __forceinline__ uint32_t mag8(const Entries<T>& e) {
  uint32_t m = Entries<T>::mag(e.w[0]);
#pragma unroll
  for (int i = 1; i < Entries<T>::kWords; ++i) m = Entries<T>::larger(m, Entries<T>::mag(e.w[i]));
  return m;
}

// Where the entries come from: X itself, or X times the slope of an activation at P.
template <typename T>
struct FromX {
  using E = Entries<T>;
  using Type = T;
  static constexpr int kRows = 8;  // rows of a tile to a thread
  // eight entries of a row from column c on, of which `left` exist
  static __device__ __forceinline__ void load(E& e, const QuantArgs& a, const T* X, long long row, long long c,
                                              long long left) {
    load8(e, X + row * a.ldx + c, left, a.unit_x);
  }
};
// Half the rows to a thread: the products are fp32 and the slopes take their time, so
// that twice the warps are worth more (8192 x 4096 bf16 with gelu: 50 us, 62 with eight
// rows; the bytes at the copy rate: 30).
template <typename T, int ACT>
struct TimesSlope {
  using E = Entries<float>;
  using Type = T;
  static constexpr int kRows = 4;
  static __device__ __forceinline__ void load(E& e, const QuantArgs& a, const T* X, long long row, long long c,
                                              long long left) {
    Entries<T> x, p;
    load8(x, X + row * a.ldx + c, left, a.unit_x);
    load8(p, static_cast<const T*>(a.P) + row * a.K + c, left, a.unit_p);
#pragma unroll
    for (int i = 0; i < 8; ++i) e.set(i, x.at(i) * slope<ACT>(p.at(i)));  // a missing entry: 0
  }
};

struct BlockScale {
  float nd, r;  // -a / 512 and the reciprocal of a / 512
};
__device__ __forceinline__ float amax_of(uint32_t bits) { return __uint_as_float(max(bits, kTinyBits)); }
__device__ __forceinline__ BlockScale block_scale(float a) {
  const float d = a * 0.001953125f;
  return BlockScale{-d, __frcp_rn(d)};
}
__device__ __forceinline__ float scale_of(float a) { return __fdiv_rn(a, 448.0f); }

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ uint64_t pmul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pfma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// Two entries to two E4M3 bytes, the first in the low byte.
__device__ __forceinline__ uint32_t quantise2(float x0, float x1, uint64_t nd, uint64_t r) {
  const uint64_t n = pmul(pair(x0, x1), pair(0.875f, 0.875f));
  const uint64_t q0 = pmul(n, r);
  const uint64_t q = pfma(pfma(q0, nd, n), r, q0);
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(q));
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
template <typename F>
__device__ __forceinline__ uint2 quantise8(F&& x, const BlockScale& b) {
  const uint64_t nd = pair(b.nd, b.nd), r = pair(b.r, b.r);
  return make_uint2(quantise2(x(0), x(1), nd, r) | (quantise2(x(2), x(3), nd, r) << 16),
                    quantise2(x(4), x(5), nd, r) | (quantise2(x(6), x(7), nd, r) << 16));
}

__device__ __forceinline__ void store8(uint8_t* p, long long left, bool vec, uint2 q) {
  if (vec && left >= 8) {
    *reinterpret_cast<uint2*>(p) = q;
  } else {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// Blocks of 128 along rows, one per half-warp (16 lanes of eight entries).
template <typename T>
__global__ void __launch_bounds__(256) quantise_rows_kernel(QuantArgs a) {
  using E = Entries<T>;
  wait_for_predecessor();
  allow_dependents();
  const long long kb = (a.K + kTile - 1) / kTile, total = a.M * kb;
  const int l16 = threadIdx.x & 15;
  const T* X = static_cast<const T*>(a.X);
  const long long b = ((long long)blockIdx.x * 256 + threadIdx.x) >> 4;
  const bool live = b < total;
  const long long row = live ? b / kb : 0, j = live ? b - row * kb : 0, c = j * kTile + l16 * 8;
  E e;
  load8(e, X + row * a.ldx + c, live ? a.K - c : 0, a.unit_x);
  uint32_t m = mag8(e);
#pragma unroll
  for (int o = 8; o; o >>= 1) m = E::larger(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (!live) return;
  const float top = amax_of(E::top(m));
  store8(a.Q + row * a.ldq + c, a.K - c, a.vec_q, quantise8([&](int i) { return e.at(i); }, block_scale(top)));
  if (l16 == 0) a.S[row * kb + j] = scale_of(top);
}

// Slot i of the blocks of 128 rows: the group's, which start at offsets[g] / 128 + g,
// and behind the last group's those of the rows that belong to none.  Every access
// stays within the matrix whatever the offsets are; all threads call this.
struct RowBlock {
  long long r0, end;
  bool rest;
};
__device__ __forceinline__ RowBlock find_block(const QuantArgs& a, long long i) {
  auto offset = [&](int g) {
    return a.wide ? static_cast<const long long*>(a.offsets)[g] : (long long)static_cast<const int*>(a.offsets)[g];
  };
  if (a.kept_offsets && blockIdx.x == 0)
    for (int g = (int)threadIdx.x; g <= a.E; g += (int)blockDim.x) a.kept_offsets[g] = offset(g);
  int before = 0;  // groups, with the rest as the last, that start at or before slot i
  for (int g0 = 0; g0 <= a.E; g0 += blockDim.x) {
    const int g = g0 + (int)threadIdx.x;
    before += __syncthreads_count(g <= a.E && offset(min(g, a.E)) / kTile + g <= i);
  }
  const int g = max(before - 1, 0);
  const long long start = offset(g), b = i - (start / kTile + g);
  RowBlock r{0, 0, g == a.E};
  if (start >= 0 && start <= a.M && b >= 0 && b <= a.M / kTile) {
    r.r0 = start + b * kTile;
    r.end = r.rest ? a.M : min(offset(g + 1), a.M);
  }
  return r;
}

// One 128 x 128 tile per block of 256 threads; a thread holds eight rows of
// eight columns (or 512 threads and four rows).  ROWS / COLS: scales along rows and along columns (with both,
// one read of X gives both results); neither: one scale for the tile.  GROUPED:
// the blocks along the columns lie in one group of rows each.  SUM: sums over the
// tile's rows, or with a.out over all rows: the blocks of a column of tiles are then
// a cluster, whose sums meet in the first's shared memory.
template <typename Src, bool ROWS, bool COLS, bool GROUPED, bool SUM>
__global__ void __launch_bounds__(16 * kTile / Src::kRows, Src::E::kPer == 2 && !SUM ? (GROUPED && ROWS ? 3 : 4) : 2)
    quantise_tile_kernel(QuantArgs a) {
  constexpr int R = Src::kRows, GRPS = kTile / R;  // rows of a thread, groups of them
  using E = typename Src::E;
  using T = typename Src::Type;
  constexpr int kWordsPerRow = kTile / E::kPer;
  __shared__ uint32_t col_mag[COLS ? GRPS : 1][kWordsPerRow];  // per group of rows
  __shared__ __align__(16) float2 col_scale[COLS ? kTile : 1];
  __shared__ __align__(16) uint8_t t_tile[COLS ? kTile * kTile : 16];  // transposed bytes, 16-byte chunks swizzled
  __shared__ uint32_t warp_mag[GRPS / 2];
  __shared__ float col_sum[SUM ? kTile : 1];
  constexpr bool TILES = !ROWS && !COLS;
  if (!TILES || !a.late) wait_for_predecessor();
  allow_dependents();
  const long long kb = (a.K + kTile - 1) / kTile, mb = GROUPED ? a.blocks : (a.M + kTile - 1) / kTile;
  long long ti = blockIdx.x / kb, tj = blockIdx.x - ti * kb;
  if constexpr (SUM) {
    if (a.out) {  // down the columns
      tj = blockIdx.x / mb;
      ti = blockIdx.x - tj * mb;
    }
  }
  const T* X = static_cast<const T*>(a.X);
  if constexpr (TILES) {  // a stack of matrices
    X += blockIdx.y * a.M * a.ldx;
    a.Q += blockIdx.y * a.M * a.ldq;
    a.S += blockIdx.y * mb * kb;
  }
  const int grp = threadIdx.x >> 4;  // rows R grp .. R grp + R - 1 of the tile
  const int l16 = threadIdx.x & 15;  // columns 8 l16 ..
  RowBlock at{ti * kTile, a.M, false};
  if constexpr (GROUPED) at = find_block(a, ti);
  const long long r0 = at.r0 + grp * R, c0 = tj * kTile + l16 * 8, left = a.K - c0;
  E e[R];
#pragma unroll
  for (int r = 0; r < R; ++r) Src::load(e[r], a, X, r0 + r, c0, r0 + r < at.end ? left : 0);

  if constexpr (TILES) {
    uint32_t m = mag8(e[0]);
#pragma unroll
    for (int r = 1; r < R; ++r) m = E::larger(m, mag8(e[r]));
    m = __reduce_max_sync(0xFFFFFFFFu, E::top(m));
    if ((threadIdx.x & 31) == 0) warp_mag[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < GRPS / 2; ++w) m = max(m, warp_mag[w]);
    const float top = amax_of(m);
    const BlockScale bs = block_scale(top);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r0 + r < a.M)
        store8(a.Q + (r0 + r) * a.ldq + c0, left, a.vec_q, quantise8([&](int i) { return e[r].at(i); }, bs));
    if (threadIdx.x == 0) a.S[ti * kb + tj] = scale_of(top);
    if (a.late) wait_for_predecessor();
    return;
  }
  if constexpr (SUM) {  // kept where the transposed bytes will be
    float* part = reinterpret_cast<float*>(t_tile) + grp * kTile + l16 * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = e[0].at(i);
#pragma unroll
      for (int r = 1; r < R; ++r) v += e[r].at(i);
      part[i] = v;
    }
  }
  if constexpr (COLS) {
#pragma unroll
    for (int w = 0; w < E::kWords; ++w) {
      uint32_t m = E::mag(e[0].w[w]);
#pragma unroll
      for (int r = 1; r < R; ++r) m = E::larger(m, E::mag(e[r].w[w]));
      col_mag[grp][l16 * E::kWords + w] = GROUPED && at.rest ? 0 : m;
    }
  }
  if constexpr (ROWS) {
    // The rows' maxima over 16 lanes: each step halves the rows a lane holds, so
    // that lane l ends up with row l R / 16's, and makes its scale.
    constexpr int SPAN = 16 / R;
    uint32_t m[R];
#pragma unroll
    for (int r = 0; r < R; ++r) m[r] = mag8(e[r]);
#pragma unroll
    for (int n = R / 2, bit = 8; n; n >>= 1, bit >>= 1) {
      const bool up = l16 & bit;
#pragma unroll
      for (int r = 0; r < n; ++r) {
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, up ? m[r] : m[r + n], bit);
        m[r] = E::larger(up ? m[r + n] : m[r], other);
      }
    }
    uint32_t mine = m[0];
#pragma unroll
    for (int bit = SPAN / 2; bit; bit >>= 1) mine = E::larger(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, bit));
    const float top = amax_of(E::top(mine));
    const BlockScale bs = block_scale(top);
    const long long my_row = r0 + l16 / SPAN;
    if (l16 % SPAN == 0 && my_row < at.end) a.S[my_row * kb + tj] = scale_of(top);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int src = (threadIdx.x & 16) + SPAN * r;
      const BlockScale rs{__shfl_sync(0xFFFFFFFFu, bs.nd, src), __shfl_sync(0xFFFFFFFFu, bs.r, src)};
      if (r0 + r < at.end)
        store8(a.Q + (r0 + r) * a.ldq + c0, left, a.vec_q, quantise8([&](int i) { return e[r].at(i); }, rs));
    }
  }
  if constexpr (COLS) {
    if constexpr (GROUPED) {
      if (ti >= mb) return;  // a slot more for the rest's rows, which are in no column block
      if (at.rest) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int w = 0; w < E::kWords; ++w) e[r].w[w] = 0;
      }
    }
    __syncthreads();
    if (threadIdx.x < kTile) {
      constexpr int kPer = E::kPer;
      const int w = threadIdx.x / kPer;
      uint32_t m = col_mag[0][w];
#pragma unroll
      for (int g = 1; g < GRPS; ++g) m = E::larger(m, col_mag[g][w]);
      // this column's of the word's entries
      if constexpr (kPer == 2) m = threadIdx.x & 1 ? m & 0xFFFF0000u : m << 16;
      const float top = amax_of(E::top(m));
      const BlockScale bs = block_scale(top);
      col_scale[threadIdx.x] = make_float2(bs.nd, bs.r);
      const long long col = tj * kTile + threadIdx.x;
      if (col < a.K) a.ST[col * mb + ti] = scale_of(top);
      if constexpr (SUM) {
        const float* part = reinterpret_cast<const float*>(t_tile) + threadIdx.x;
        float v = part[0];
#pragma unroll
        for (int g = 1; g < GRPS; ++g) v += part[g * kTile];
        if (a.out) col_sum[threadIdx.x] = v;
        else if (col < a.K) a.sums[ti * a.K + col] = v;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = l16 * 8 + i;
      const float2 cs = col_scale[c];
      // column c's 128 bytes are a row of t_tile; this thread's R bytes lie in its 16-byte chunk grp R / 16
      const int chunk = (grp * R >> 4) ^ (l16 & 7);
      uint8_t* dst = &t_tile[c * kTile + chunk * 16 + (grp * R & 15)];
      const BlockScale bs{cs.x, cs.y};
      if constexpr (R == 8) {
        *reinterpret_cast<uint2*>(dst) = quantise8([&](int r) { return e[r].at(i); }, bs);
      } else {
        const uint64_t nd = pair(bs.nd, bs.nd), rr = pair(bs.r, bs.r);
        *reinterpret_cast<uint32_t*>(dst) =
            quantise2(e[0].at(i), e[1].at(i), nd, rr) | (quantise2(e[2].at(i), e[3].at(i), nd, rr) << 16);
      }
    }
    __syncthreads();
    const int j = threadIdx.x & 7;  // 16-byte chunk: rows 16 j of the tile
    const long long limit = GROUPED ? a.blocks * kTile : a.M;
#pragma unroll
    for (int p = 0; p < R / 2; ++p) {
      const int c = p * 2 * GRPS + (threadIdx.x >> 3);
      const long long col = tj * kTile + c, row = ti * kTile + 16 * j;
      if (col < a.K && row < limit) {
        const uint4 q = *reinterpret_cast<const uint4*>(&t_tile[c * kTile + ((j ^ ((c >> 3) & 7)) * 16)]);
        uint8_t* out = a.QT + col * a.ldqt + row;
        if (a.vec_qt && limit - row >= 16) {
          *reinterpret_cast<uint4*>(out) = q;
        } else {
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
          for (int i = 0; i < 16; ++i)
            if (row + i < limit) out[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
        }
      }
    }
    if constexpr (SUM) {
      if (a.out) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        const long long col = tj * kTile + threadIdx.x;
        if (ti == 0 && threadIdx.x < kTile && col < a.K) {
          const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&col_sum[threadIdx.x]);
          float v = col_sum[threadIdx.x];
          for (int r = 1; r < (int)mb; ++r) {
            uint32_t at;
            float w;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(r));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(at) : "memory");
            v += w;
          }
          store_real(a.out, a.out_type, col, v);
        }
        __syncwarp();  // none leaves while its sums are read
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
      }
    }
  }
}

// Eight rows of threads each add every eighth partial sum of 32 columns, then the
// eight meet in order.
__global__ void __launch_bounds__(256) sum_rows_kernel(const float* sums, long long rows, long long K, void* out,
                                                       int type) {
  __shared__ float part[8][32];
  wait_for_predecessor();
  allow_dependents();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const long long col = (long long)blockIdx.x * 32 + x;
  float v = 0.0f;
  if (col < K)
    for (long long r = y; r < rows; r += 8) v += sums[r * K + col];
  part[y][x] = v;
  __syncthreads();
  if (y == 0 && col < K) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += part[i][x];
    store_real(out, type, col, v);
  }
}

// A kernel with column sums: in clusters down the columns where one holds them all.
template <typename Src>
cudaError_t launch_sums(QuantArgs a, dim3 g, dim3 b, cudaStream_t st) {
  const auto kernel = quantise_tile_kernel<Src, true, true, false, true>;
  const long long mb = (a.M + kTile - 1) / kTile;
  if (!a.out || mb > kSumCluster) {
    a.out = nullptr;
    return launch_dependent(kernel, g, b, 0, st, a);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = g;
  cfg.blockDim = b;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)mb;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename Src>
cudaError_t launch_tiles(const QuantArgs& a, int form, dim3 g, cudaStream_t st) {
  const dim3 b(256);
  if (a.offsets)
    return form == RG_F8_COLUMNS
               ? launch_dependent(quantise_tile_kernel<Src, false, true, true, false>, g, b, 0, st, a)
               : launch_dependent(quantise_tile_kernel<Src, true, true, true, false>, g, b, 0, st, a);
  switch (form) {
    case RG_F8_ROWS: return launch_dependent(quantise_tile_kernel<Src, true, false, false, false>, g, b, 0, st, a);
    case RG_F8_COLUMNS: return launch_dependent(quantise_tile_kernel<Src, false, true, false, false>, g, b, 0, st, a);
    case RG_F8_BOTH:
      return a.sums ? launch_sums<Src>(a, g, b, st)
                    : launch_dependent(quantise_tile_kernel<Src, true, true, false, false>, g, b, 0, st, a);
    default: return launch_dependent(quantise_tile_kernel<Src, false, false, false, false>, g, b, 0, st, a);
  }
}
// With an activation's slope: form both, with the column sums where they are wanted.
template <typename T, int ACT>
cudaError_t launch_slope(const QuantArgs& a, dim3 g, cudaStream_t st) {
  using Src = TimesSlope<T, ACT>;
  const dim3 b(16 * kTile / Src::kRows);
  return a.sums ? launch_sums<Src>(a, g, b, st)
                : launch_dependent(quantise_tile_kernel<Src, true, true, false, false>, g, b, 0, st, a);
}

template <typename T>
cudaError_t launch_t(const QuantArgs& a, int form, cudaStream_t st) {
  const long long kb = (a.K + kTile - 1) / kTile;
  // groups with their rows: a slot more for those behind the last group
  const long long mb = a.offsets ? a.blocks + (form == RG_F8_BOTH) : (a.M + kTile - 1) / kTile;
  // Along rows: up to 2^15 blocks of 128, or fewer rows than half a tile, go a
  // block to a half-warp, which spreads few blocks over more SMs (512 x 1024:
  // 2.1 us, in tiles 3.0); more go in tiles, where a thread has eight loads on
  // its way (8192 x 4096 bf16: 26 us a block to a half-warp).
  const bool tiles = form != RG_F8_ROWS || (a.M >= 64 && a.M * kb > (1LL << 15));
  const long long blocks = tiles ? mb * kb : (a.M * kb + 15) / 16;
  if (blocks > INT_MAX || a.batch > 65535) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)blocks, (unsigned)a.batch);
  if (!tiles) return launch_dependent(quantise_rows_kernel<T>, g, dim3(256), 0, st, a);
  switch (a.act) {
    case RG_ACT_RELU: return launch_slope<T, RG_ACT_RELU>(a, g, st);
    case RG_ACT_SILU: return launch_slope<T, RG_ACT_SILU>(a, g, st);
    case RG_ACT_GELU: return launch_slope<T, RG_ACT_GELU>(a, g, st);
    case RG_ACT_GELU_TANH: return launch_slope<T, RG_ACT_GELU_TANH>(a, g, st);
    default: return launch_tiles<FromX<T>>(a, form, g, st);
  }
}

}  // namespace

cudaError_t launch_sum_rows(const float* sums, long long rows, long long K, void* out, int type, cudaStream_t st) {
  return launch_dependent(sum_rows_kernel, dim3((unsigned)((K + 31) / 32)), dim3(256), 0, st, sums, rows, K, out, type);
}

cudaError_t launch_quantise_f8(QuantArgs a, int type, int form, cudaStream_t st) {
  const size_t es = type == RG_TYPE_F32 ? 4 : 2;
  auto aligned = [](const void* p, long long row_bytes, unsigned n) {
    return (reinterpret_cast<uintptr_t>(p) % n) == 0 && row_bytes % n == 0;
  };
  a.unit_x = row_unit(a.X, a.ldx * (long long)es);
  a.unit_p = row_unit(a.P, a.K * (long long)es);
  a.vec_q = aligned(a.Q, a.ldq, 8);
  a.vec_qt = aligned(a.QT, a.ldqt, 16);
  switch (type) {
    case RG_TYPE_F32: return launch_t<float>(a, form, st);
    case RG_TYPE_F16: return launch_t<__half>(a, form, st);
    default: return launch_t<__nv_bfloat16>(a, form, st);
  }
}

}  // namespace rg
