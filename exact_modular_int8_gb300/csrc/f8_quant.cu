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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <climits>
#include <cstdint>

#include "f8_kernels.h"

namespace rg {
namespace {

constexpr uint32_t kTinyBits = 0x21800000u;  // 2^-60
constexpr int kTile = 128;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Magnitudes are compared as bit patterns: the order of the non-negative
// floats, with NaN above inf, so that a NaN is never lost.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct BlockScale {
  float d, r;  // a / 512 and its reciprocal
  float s;     // a / 448
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  const float a = __uint_as_float(max(amax_bits, kTinyBits));
  BlockScale b;
  b.d = a * 0.001953125f;
  b.r = __frcp_rn(b.d);
  b.s = __fdiv_rn(a, 448.0f);
  return b;
}
__device__ __forceinline__ float scaled(float x, float d, float r) {
  const float n = x * 0.875f;
  const float q0 = n * r;
  return __fmaf_rn(__fmaf_rn(-q0, d, n), r, q0);
}
// Two values to two E4M3 bytes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Eight entries of a row from column c (limit: entries left in the row);
// missing ones read as 0.
template <typename T>
__device__ __forceinline__ void load8(const T* p, long long left, bool vec, float (&v)[8]) {
  if (vec && left >= 8) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const unsigned short h = (unsigned short)(w[i >> 1] >> (16 * (i & 1)));
        v[i] = to_f32(*reinterpret_cast<const T*>(&h));
      }
    } else {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : 0.0f;
  }
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

__device__ __forceinline__ uint2 quantise8(const float (&v)[8], const BlockScale& b) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = scaled(v[i], b.d, b.r);
  return make_uint2(e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16), e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16));
}

// One block of 128 per half-warp: 16 lanes of eight entries.
template <typename T>
__global__ void __launch_bounds__(256) quantise_rows_kernel(QuantArgs a) {
  const long long kb = (a.K + kTile - 1) / kTile, total = a.M * kb;
  const int lane16 = threadIdx.x & 15;
  const T* X = static_cast<const T*>(a.X);
  const long long b = ((long long)blockIdx.x * 256 + threadIdx.x) >> 4;
  const bool live = b < total;
  const long long row = live ? b / kb : 0, j = live ? b - row * kb : 0;
  const long long c = j * kTile + lane16 * 8, left = live ? a.K - c : 0;
  float v[8];
  load8(X + row * a.ldx + c, left, a.vec_x, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag(v[i]));
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (!live) return;
  const BlockScale bs = block_scale(m);
  store8(a.Q + row * a.ldq + c, left, a.vec_q, quantise8(v, bs));
  if (lane16 == 0) a.S[row * kb + j] = bs.s;
}

// One 128 x 128 tile per block of 256 threads; a thread holds eight rows of
// eight columns.  ROWS / COLS: scales along rows and along columns (with both,
// one read of X gives both results); neither: one scale for the tile.
template <typename T, bool ROWS, bool COLS>
__global__ void __launch_bounds__(256) quantise_tile_kernel(QuantArgs a) {
  __shared__ uint32_t col_max[16][kTile];           // per 8-row group
  __shared__ __align__(16) uint8_t t_tile[COLS ? kTile * kTile : 16];  // transposed bytes, 16-byte chunks swizzled
  __shared__ uint32_t warp_max[8];
  const long long kb = (a.K + kTile - 1) / kTile, mb = (a.M + kTile - 1) / kTile;
  const long long ti = blockIdx.x / kb, tj = blockIdx.x - ti * kb;
  const T* X = static_cast<const T*>(a.X);
  const int grp = threadIdx.x >> 4;   // rows 8 grp .. 8 grp + 7 of the tile
  const int l16 = threadIdx.x & 15;   // columns 8 l16 ..
  const long long r0 = ti * kTile + grp * 8, c0 = tj * kTile + l16 * 8, left = a.K - c0;
  float v[8][8];
#pragma unroll
  for (int r = 0; r < 8; ++r) load8(X + (r0 + r) * a.ldx + c0, r0 + r < a.M ? left : 0, a.vec_x, v[r]);

  if constexpr (!ROWS && !COLS) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, mag(v[r][i]));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, warp_max[w]);
    const BlockScale bs = block_scale(m);
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (r0 + r < a.M) store8(a.Q + (r0 + r) * a.ldq + c0, left, a.vec_q, quantise8(v[r], bs));
    if (threadIdx.x == 0) a.S[ti * kb + tj] = bs.s;
    return;
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, mag(v[r][i]));
#pragma unroll
      for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const BlockScale bs = block_scale(m);
      if (r0 + r < a.M) {
        store8(a.Q + (r0 + r) * a.ldq + c0, left, a.vec_q, quantise8(v[r], bs));
        if (l16 == 0) a.S[(r0 + r) * kb + tj] = bs.s;
      }
    }
  }
  if constexpr (COLS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < 8; ++r) m = max(m, mag(v[r][i]));
      col_max[grp][l16 * 8 + i] = m;
    }
    __syncthreads();
    if (threadIdx.x < kTile) {
      uint32_t m = 0;
#pragma unroll
      for (int g = 0; g < 16; ++g) m = max(m, col_max[g][threadIdx.x]);
      col_max[0][threadIdx.x] = m;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = l16 * 8 + i;
      const BlockScale bs = block_scale(col_max[0][c]);
      float w[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) w[r] = v[r][i];
      // column c's 128 bytes are a row of t_tile; this thread's 8 bytes are half of its 16-byte chunk grp / 2
      const int chunk = (grp >> 1) ^ (l16 & 7);
      *reinterpret_cast<uint2*>(&t_tile[c * kTile + chunk * 16 + (grp & 1) * 8]) = quantise8(w, bs);
    }
    if (threadIdx.x < kTile && tj * kTile + threadIdx.x < a.K)
      a.ST[(tj * kTile + threadIdx.x) * mb + ti] = block_scale(col_max[0][threadIdx.x]).s;
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
  const long long blocks = form == RG_F8_ROWS ? (a.M * kb + 15) / 16 : mb * kb;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)blocks), b(256);
  switch (form) {
    case RG_F8_ROWS: quantise_rows_kernel<T><<<g, b, 0, st>>>(a); break;
    case RG_F8_COLUMNS: quantise_tile_kernel<T, false, true><<<g, b, 0, st>>>(a); break;
    case RG_F8_BOTH: quantise_tile_kernel<T, true, true><<<g, b, 0, st>>>(a); break;
    default: quantise_tile_kernel<T, false, false><<<g, b, 0, st>>>(a); break;
  }
  return cudaGetLastError();
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
