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
  __device__ __forceinline__ void set(int i, float v) { w[i] = __float_as_uint(v); }
  static __device__ __forceinline__ uint32_t mag(uint32_t a) { return a & 0x7FFFFFFFu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
  static __device__ __forceinline__ uint32_t top(uint32_t m) { return m; }
};

// Eight entries from p, of which `left` exist; missing ones read as 0.
template <typename T>
__device__ __forceinline__ void load8(Entries<T>& e, const T* p, long long left, bool vec) {
  if (vec && left >= 8) {
    e.load(p);
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
  load8(e, X + row * a.ldx + c, live ? a.K - c : 0, a.vec_x);
  uint32_t m = mag8(e);
#pragma unroll
  for (int o = 8; o; o >>= 1) m = E::larger(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (!live) return;
  const float top = amax_of(E::top(m));
  store8(a.Q + row * a.ldq + c, a.K - c, a.vec_q, quantise8([&](int i) { return e.at(i); }, block_scale(top)));
  if (l16 == 0) a.S[row * kb + j] = scale_of(top);
}

// One 128 x 128 tile per block of 256 threads; a thread holds eight rows of
// eight columns.  ROWS / COLS: scales along rows and along columns (with both,
// one read of X gives both results); neither: one scale for the tile.
template <typename T, bool ROWS, bool COLS>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) quantise_tile_kernel(QuantArgs a) {
  using E = Entries<T>;
  constexpr int kWordsPerRow = kTile / E::kPer;
  __shared__ uint32_t col_mag[COLS ? 16 : 1][kWordsPerRow];  // per 8-row group
  __shared__ __align__(16) float2 col_scale[COLS ? kTile : 1];
  __shared__ __align__(16) uint8_t t_tile[COLS ? kTile * kTile : 16];  // transposed bytes, 16-byte chunks swizzled
  __shared__ uint32_t warp_mag[8];
  wait_for_predecessor();
  allow_dependents();
  const long long kb = (a.K + kTile - 1) / kTile, mb = (a.M + kTile - 1) / kTile;
  const long long ti = blockIdx.x / kb, tj = blockIdx.x - ti * kb;
  const T* X = static_cast<const T*>(a.X);
  const int grp = threadIdx.x >> 4;  // rows 8 grp .. 8 grp + 7 of the tile
  const int l16 = threadIdx.x & 15;  // columns 8 l16 ..
  const long long r0 = ti * kTile + grp * 8, c0 = tj * kTile + l16 * 8, left = a.K - c0;
  E e[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) load8(e[r], X + (r0 + r) * a.ldx + c0, r0 + r < a.M ? left : 0, a.vec_x);

  if constexpr (!ROWS && !COLS) {
    uint32_t m = mag8(e[0]);
#pragma unroll
    for (int r = 1; r < 8; ++r) m = E::larger(m, mag8(e[r]));
    m = __reduce_max_sync(0xFFFFFFFFu, E::top(m));
    if ((threadIdx.x & 31) == 0) warp_mag[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, warp_mag[w]);
    const float top = amax_of(m);
    const BlockScale bs = block_scale(top);
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (r0 + r < a.M)
        store8(a.Q + (r0 + r) * a.ldq + c0, left, a.vec_q, quantise8([&](int i) { return e[r].at(i); }, bs));
    if (threadIdx.x == 0) a.S[ti * kb + tj] = scale_of(top);
    return;
  }
  if constexpr (COLS) {
#pragma unroll
    for (int w = 0; w < E::kWords; ++w) {
      uint32_t m = E::mag(e[0].w[w]);
#pragma unroll
      for (int r = 1; r < 8; ++r) m = E::larger(m, E::mag(e[r].w[w]));
      col_mag[grp][l16 * E::kWords + w] = m;
    }
  }
  if constexpr (ROWS) {
    // The eight rows' maxima over 16 lanes: each step halves the rows a lane
    // holds, so that lane l ends up with row l / 2's, and makes its scale.
    uint32_t m[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) m[r] = mag8(e[r]);
#pragma unroll
    for (int n = 4, bit = 8; n; n >>= 1, bit >>= 1) {
      const bool up = l16 & bit;
#pragma unroll
      for (int r = 0; r < n; ++r) {
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, up ? m[r] : m[r + n], bit);
        m[r] = E::larger(up ? m[r + n] : m[r], other);
      }
    }
    const uint32_t mine = E::larger(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
    const float top = amax_of(E::top(mine));
    const BlockScale bs = block_scale(top);
    const long long my_row = r0 + (l16 >> 1);
    if (!(l16 & 1) && my_row < a.M) a.S[my_row * kb + tj] = scale_of(top);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int src = (threadIdx.x & 16) + 2 * r;
      const BlockScale rs{__shfl_sync(0xFFFFFFFFu, bs.nd, src), __shfl_sync(0xFFFFFFFFu, bs.r, src)};
      if (r0 + r < a.M)
        store8(a.Q + (r0 + r) * a.ldq + c0, left, a.vec_q, quantise8([&](int i) { return e[r].at(i); }, rs));
    }
  }
  if constexpr (COLS) {
    __syncthreads();
    if (threadIdx.x < kTile) {
      constexpr int kPer = E::kPer;
      const int w = threadIdx.x / kPer;
      uint32_t m = col_mag[0][w];
#pragma unroll
      for (int g = 1; g < 16; ++g) m = E::larger(m, col_mag[g][w]);
      // this column's of the word's entries
      if constexpr (kPer == 2) m = threadIdx.x & 1 ? m & 0xFFFF0000u : m << 16;
      const float top = amax_of(E::top(m));
      const BlockScale bs = block_scale(top);
      col_scale[threadIdx.x] = make_float2(bs.nd, bs.r);
      const long long col = tj * kTile + threadIdx.x;
      if (col < a.K) a.ST[col * mb + ti] = scale_of(top);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = l16 * 8 + i;
      const float2 cs = col_scale[c];
      // column c's 128 bytes are a row of t_tile; this thread's 8 bytes are half of its 16-byte chunk grp / 2
      const int chunk = (grp >> 1) ^ (l16 & 7);
      *reinterpret_cast<uint2*>(&t_tile[c * kTile + chunk * 16 + (grp & 1) * 8]) =
          quantise8([&](int r) { return e[r].at(i); }, BlockScale{cs.x, cs.y});
    }
    __syncthreads();
    const int j = threadIdx.x & 7;  // 16-byte chunk: rows 16 j of the tile
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int c = p * 32 + (threadIdx.x >> 3);
      const long long col = tj * kTile + c, row = ti * kTile + 16 * j;
      if (col < a.K && row < a.M) {
        const uint4 q = *reinterpret_cast<const uint4*>(&t_tile[c * kTile + ((j ^ ((c >> 3) & 7)) * 16)]);
        uint8_t* out = a.QT + col * a.ldqt + row;
        if (a.vec_qt && a.M - row >= 16) {
          *reinterpret_cast<uint4*>(out) = q;
        } else {
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
          for (int i = 0; i < 16; ++i)
            if (row + i < a.M) out[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const QuantArgs& a, int form, cudaStream_t st) {
  const long long kb = (a.K + kTile - 1) / kTile, mb = (a.M + kTile - 1) / kTile;
  // Along rows: up to 2^15 blocks of 128, or fewer rows than half a tile, go a
  // block to a half-warp, which spreads few blocks over more SMs (512 x 1024:
  // 2.1 us, in tiles 3.0); more go in tiles, where a thread has eight loads on
  // its way (8192 x 4096 bf16: 26 us a block to a half-warp).
  const bool tiles = form != RG_F8_ROWS || (a.M >= 64 && a.M * kb > (1LL << 15));
  const long long blocks = tiles ? mb * kb : (a.M * kb + 15) / 16;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)blocks), b(256);
  if (!tiles) {
    return launch_dependent(quantise_rows_kernel<T>, g, b, 0, st, a);
  }
  switch (form) {
    case RG_F8_ROWS: return launch_dependent(quantise_tile_kernel<T, true, false>, g, b, 0, st, a);
    case RG_F8_COLUMNS: return launch_dependent(quantise_tile_kernel<T, false, true>, g, b, 0, st, a);
    case RG_F8_BOTH: return launch_dependent(quantise_tile_kernel<T, true, true>, g, b, 0, st, a);
    default: return launch_dependent(quantise_tile_kernel<T, false, false>, g, b, 0, st, a);
  }
}

}  // namespace

cudaError_t launch_quantise_f8(QuantArgs a, int type, int form, cudaStream_t st) {
  const size_t es = type == RG_TYPE_F32 ? 4 : 2;
  auto aligned = [](const void* p, long long row_bytes, unsigned n) {
    return (reinterpret_cast<uintptr_t>(p) % n) == 0 && row_bytes % n == 0;
  };
  a.vec_x = aligned(a.X, a.ldx * (long long)es, 16);
  a.vec_q = aligned(a.Q, a.ldq, 8);
  a.vec_qt = aligned(a.QT, a.ldqt, 16);
  switch (type) {
    case RG_TYPE_F32: return launch_t<float>(a, form, st);
    case RG_TYPE_F16: return launch_t<__half>(a, form, st);
    default: return launch_t<__nv_bfloat16>(a, form, st);
  }
}

}  // namespace rg
