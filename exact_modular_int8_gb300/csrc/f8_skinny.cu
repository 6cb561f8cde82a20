// f8_skinny.cu -- block-scaled E4M3 products with at most 32 rows of A (decoding).
//
// With few rows the work is reading B once.  B's rows are the 16-row operand of
// warp-level MMAs (m16n8k16) and A's rows their columns, so nothing is padded
// to the 128 rows of a tcgen05 tile.  The operands enter as fp16, in which E4M3
// is exact, with fp32 sums.  The MMA's order of k is free as long as both
// operands agree: a lane loads 16 consecutive bytes of a row, which feed four
// MMAs without a shuffle.
//
// A tile is 16 MT rows of B over all of K, a block's eight warps taking every
// eighth 128-block each; the blocks (two per SM with one column tile) walk the
// tiles.  What a warp needs of one 128-block -- B's and A's rows and the scales --
// is a piece, copied to shared memory (cp.async) kRing - 1 pieces ahead of its
// use and across tiles.  The warps' sums meet in shared memory in a fixed order.
//
// Bound by memory and, for short calls, by its latency: one row of 4096 x 2048 in
// 3.0 us (the bytes alone take 1.25), of 8192 x 4096 in 8.7 us (5.0), of 70000 x
// 4096 in 52 us (5.5 TB/s), one launch after another.  Before the copies (loads to
// registers, a tile per block) the second took 2 us more.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "f8_kernels.h"

namespace rg {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

struct SkinnyParams {
  const uint8_t* A;
  const uint8_t* B;
  const float* SA;
  const float* SB;
  void* C;
  long long lda, ldb, ldc, sb_n;
  int M, N, K, KB;
  int tiles;
  int out_type;
  int keep_status;
  DevPlan* plan;
};

__device__ __forceinline__ uint32_t h2_of_e4m3x2(uint32_t two) {  // the low 16 bits: two E4M3 values
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes of which the first n exist; the others become zeros and are not read.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float lds4(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

template <int NT, int MT>
struct Shape {
  static constexpr int kRing = NT == 1 ? 4 : 3;
  static constexpr int kRows = 16 * MT + 8 * NT;           // of B, then of A: 128 bytes each
  static constexpr int kScales = kRows * 128;              // offset of the scales, in the rows' order
  static constexpr int kPiece = kScales + kRows * 4;       // a multiple of 16
  static constexpr int kLd = 8 * NT + 4;                   // a row of the warps' sums, padded
  static constexpr int kRed = kWarps * 16 * MT * kLd * 4;  // twice: tiles alternate
  static constexpr int kSmem = 2 * kRed + kWarps * kRing * kPiece;
};

template <int NT, int MT, bool TILE_B>
__global__ void __launch_bounds__(kThreads) f8_skinny_kernel(const __grid_constant__ SkinnyParams p) {
  using S = Shape<NT, MT>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  wait_for_predecessor();
  allow_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0 && !p.keep_status) {  // no wait here that could fail
    p.plan->status = 0;
    p.plan->timeout_where = 0;
  }
  const uint32_t ring = su32(smem) + 2 * S::kRed + warp * S::kRing * S::kPiece;

  // Copies of the next piece: 128-block pkb of tile pt.  Row r's 16-byte chunk c
  // lies at r * 128 + (c ^ 4 (r & 1)) * 16, which the MMA lanes read without bank
  // conflicts; eight lanes copy a whole 128-byte line.  Rows of B past the last
  // repeat it, rows of A past the last are left out: their results are not stored.
  int pt = blockIdx.x, pkb = warp;
  auto copy_next = [&](int slot) {
    if (pt < p.tiles && pkb < p.KB) {
      const uint32_t at = ring + slot * S::kPiece;
      const int c = lane & 7, k = pkb * 128 + c * 16, n = min(max(p.K - k, 0), 16);
      const uint32_t dst = at + (lane >> 3) * 128 + ((c ^ (((lane >> 3) & 1) << 2)) << 4);
#pragma unroll
      for (int r0 = 0; r0 < 16 * MT; r0 += 4) {
        const int row = min(pt * 16 * MT + r0 + (lane >> 3), p.N - 1);
        copy16(dst + r0 * 128, p.B + (long long)row * p.ldb + (n ? k : 0), n);
      }
#pragma unroll
      for (int r0 = 0; r0 < 8 * NT; r0 += 4) {
        const int row = r0 + (lane >> 3);
        if (row < p.M) copy16(dst + (16 * MT + r0) * 128, p.A + (long long)row * p.lda + (n ? k : 0), n);
      }
      for (int r = lane; r < S::kRows; r += 32) {
        if (r < 16 * MT) {
          const int row = min(pt * 16 * MT + r, p.N - 1);
          if (!TILE_B || r == 0) copy4(at + S::kScales + r * 4, p.SB + (long long)(TILE_B ? row / 128 : row) * p.sb_n + pkb);
        } else if (r - 16 * MT < p.M) {
          copy4(at + S::kScales + r * 4, p.SA + (long long)(r - 16 * MT) * p.KB + pkb);
        }
      }
      pkb += kWarps;
      if (pkb >= p.KB) {
        pkb = warp;
        pt += gridDim.x;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < S::kRing - 1; ++s) copy_next(s);

  int slot = 0, parity = 0;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, parity ^= 1) {
    float tot[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) tot[m][i][0] = tot[m][i][1] = tot[m][i][2] = tot[m][i][3] = 0.0f;
    for (int kb = warp; kb < p.KB; kb += kWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S::kRing - 2) : "memory");
      __syncwarp();
      const uint32_t piece = ring + slot * S::kPiece;
      float acc[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.0f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t at = piece + g * 128 + (((half * 4 + t4) ^ ((g & 1) << 2)) << 4);
        uint4 a[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) a[i] = lds16(at + (16 * MT + 8 * i) * 128);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint4 lo = lds16(at + 16 * m * 128), hi = lds16(at + (16 * m + 8) * 128);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // four of the lane's 16 values of k
            const uint32_t l = word(lo, j), h = word(hi, j);
            const uint32_t w[4] = {h2_of_e4m3x2(l), h2_of_e4m3x2(h), h2_of_e4m3x2(l >> 16), h2_of_e4m3x2(h >> 16)};
#pragma unroll
            for (int i = 0; i < NT; ++i)
              mma16816(acc[m][i], w, h2_of_e4m3x2(word(a[i], j)), h2_of_e4m3x2(word(a[i], j) >> 16));
          }
        }
      }
      float sa[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) sa[i][c] = lds4(piece + S::kScales + (16 * MT + 8 * i + 2 * t4 + c) * 4);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float sb = lds4(piece + S::kScales + (TILE_B ? 0 : 16 * m + 8 * h + g) * 4);
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              tot[m][i][2 * h + c] = fmaf(acc[m][i][2 * h + c], sb * sa[i][c], tot[m][i][2 * h + c]);
        }
      // the slot before this one: all lanes have read it since they met above
      copy_next(slot == 0 ? S::kRing - 1 : slot - 1);
      slot = slot + 1 == S::kRing ? 0 : slot + 1;
    }
    float* red = reinterpret_cast<float*>(smem + parity * S::kRed);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(&red[((warp * MT + m) * 16 + 8 * h + g) * S::kLd + 8 * i + 2 * t4]) =
              make_float2(tot[m][i][2 * h], tot[m][i][2 * h + 1]);
    __syncthreads();  // the next tile's sums go to the other buffer
    for (int o = threadIdx.x; o < 16 * MT * p.M; o += kThreads) {
      const int m = o / (16 * MT), r = o - m * 16 * MT, n = tile * 16 * MT + r;
      if (n >= p.N) continue;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += red[(w * MT * 16 + r) * S::kLd + m];
      const long long at = (long long)m * p.ldc + n;
      if (p.out_type == RG_TYPE_F32) static_cast<float*>(p.C)[at] = v;
      else if (p.out_type == RG_TYPE_F16) static_cast<__half*>(p.C)[at] = __float2half_rn(v);
      else static_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(v);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// The kernel's blocks per SM times the SMs of this device, found once.
template <int NT, int MT, bool TILE_B>
cudaError_t launch(SkinnyParams p, cudaStream_t st) {
  using S = Shape<NT, MT>;
  static_assert(S::kSmem <= 232448 && S::kPiece % 16 == 0 && S::kRed % 16 == 0, "shared memory");
  static std::atomic<int> blocks[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int resident = blocks[dev].load(std::memory_order_relaxed);
  if (!resident) {
    int sms = 0, per_sm = 0;
    e = cudaFuncSetAttribute(f8_skinny_kernel<NT, MT, TILE_B>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, f8_skinny_kernel<NT, MT, TILE_B>, kThreads, S::kSmem);
    if (e != cudaSuccess) return e;
    resident = sms * std::max(per_sm, 1);
    blocks[dev].store(resident, std::memory_order_relaxed);
  }
  p.tiles = (p.N + 16 * MT - 1) / (16 * MT);
  return launch_dependent(f8_skinny_kernel<NT, MT, TILE_B>, dim3((unsigned)std::min(p.tiles, resident)),
                          dim3(kThreads), S::kSmem, st, p);
}

template <int NT, int MT>
cudaError_t launch(const SkinnyParams& p, bool tile_b, cudaStream_t st) {
  return tile_b ? launch<NT, MT, true>(p, st) : launch<NT, MT, false>(p, st);
}

}  // namespace

cudaError_t launch_f8_skinny(const F8GemmArgs& a, DevPlan* plan, cudaStream_t st) {
  const SkinnyParams p{a.A, a.B, a.SA, a.SB, a.C, a.lda, a.ldb, a.ldc, a.sb_n, (int)a.M, (int)a.N, (int)a.K,
                       (int)((a.K + 127) / 128), 0, a.out_type, a.keep_status, plan};
  // with more than eight rows, two row tiles of B share a piece's rows of A
  if (a.M <= 8) return launch<1, 1>(p, a.tile_b, st);
  if (a.M <= 16) return launch<2, 2>(p, a.tile_b, st);
  if (a.M <= 24) return launch<3, 1>(p, a.tile_b, st);
  return launch<4, 1>(p, a.tile_b, st);
}

}  // namespace rg
