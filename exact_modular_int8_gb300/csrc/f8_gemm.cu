// f8_gemm.cu -- products of block-scaled E4M3 matrices on the sm_103a tensor cores.
//
//   C[m][n] = sum_kb sa[m][kb] sb[n][kb] P_kb[m][n],  P_kb = A_kb B_kb^T over 128 values of k
//
// tcgen05.mma kind::f8f6f4 forms P_kb in tensor memory (fp32): four MMAs of
// K = 32 per block, since the scales are general fp32 numbers the tensor core
// cannot apply.  The epilogue warps read every P_kb back and add it, scaled,
// to fp32 sums in registers, so the scaling costs one fused multiply-add per
// entry and block (one more multiplication when both sides scale per entry of
// the block's row), beside the MMAs of the next block: two accumulators
// alternate.
//
// Warp roles: warp 0 TMA producer, warp 1 tensor memory and MMA issue, warps
// 2..9 epilogue.  Every wait is bounded as in the residue product.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "f8_kernels.h"
#include "rg_tc.cuh"

namespace rg {
namespace {

constexpr int BK = 128;  // values of k per block and pipeline stage: one 128-byte swizzle row
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 64 + 32 * EPI_WARPS;
constexpr int SLAB = 128 * BK;  // 128 rows (or columns) of one stage

// Instruction descriptor, kind::f8f6f4: D f32, A and B E4M3, A K-major.
__host__ __device__ constexpr uint32_t idesc_f8(int m, int n, bool b_kmajor) {
  return (1u << 4) | (b_kmajor ? 0u : 1u << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

struct Params {
  const float* SA;
  const float* SB;
  void* C;
  long long ldc, sb_n, sb_k;
  int M, N, KB;
  int mt, nt;
  int out_type;
  int vec_c;  // rows of C start on 16-byte boundaries
  int fault;
  unsigned long long wait_ns;
};

__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ void store_out(void* C, long long at, int type, float v) {
  if (type == RG_TYPE_F32) static_cast<float*>(C)[at] = v;
  else if (type == RG_TYPE_F16) static_cast<__half*>(C)[at] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(C)[at] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------------------
// Tiles of 128 x 128, one per cluster of S CTAs: each CTA sums a slice of K,
// and the slices are joined through distributed shared memory in rank order.
// ---------------------------------------------------------------------------
constexpr int BN1 = 128;
constexpr int STAGES1 = 6;
constexpr int STAGE1_BYTES = 2 * SLAB;
constexpr int PART_LD = BN1 + 4;  // floats per row of a CTA's partial tile, kept where the stages were
static_assert(128 * PART_LD * 4 <= STAGES1 * STAGE1_BYTES, "partial tile");
constexpr int SCALE1_BYTES = EPI_WARPS * 2 * 64 * 4;
constexpr int SMEM1_BYTES = 1024 + STAGES1 * STAGE1_BYTES + SCALE1_BYTES + 256;
static_assert(SMEM1_BYTES <= 232448, "shared memory");

template <bool B_KMAJOR, bool TILE_B>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    f8_gemm_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ Params gp, int S, DevPlan* plan) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stage_base = smem;
  float* scale_base = reinterpret_cast<float*>(smem + STAGES1 * STAGE1_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES1 * STAGE1_BYTES + SCALE1_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = bars + STAGES1;
  uint64_t* tfull = bars + 2 * STAGES1;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tfull + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x % (unsigned)S), tile = (int)(blockIdx.x / (unsigned)S);
  const int tn = tile / gp.mt, tm = tile - tn * gp.mt;
  const int kbs = (gp.KB + S - 1) / S;
  const int kb_lo = min(rank * kbs, gp.KB), kb_hi = min(kb_lo + kbs, gp.KB);
  Ctl ctl{abort_flag, &plan->status, &plan->timeout_where, gp.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES1; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), EPI_WARPS);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"((uint32_t)(2 * BN1)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  wait_for_predecessor();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool issued[STAGES1] = {};
      uint32_t issued_phase[STAGES1] = {};
      bool ok = true;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!wait_bounded(smem_u32(&empty[stage]), phase ^ 1u, ctl, 21)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&full[stage]);
        mbar_arrive_expect_tx(fb, STAGE1_BYTES);
        const uint32_t a_dst = smem_u32(stage_base + stage * STAGE1_BYTES);
        tma_load_2d(a_dst, &tmA, fb, kb * BK, tm * 128);
        if constexpr (B_KMAJOR) tma_load_2d(a_dst + SLAB, &tmB, fb, kb * BK, tn * BN1);
        else tma_load_2d(a_dst + SLAB, &tmB, fb, tn * BN1, kb * BK);
        issued[stage] = true;
        issued_phase[stage] = phase;
        if (++stage == STAGES1) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {  // let issued copies land before the block exits
        Ctl drain_ctl = ctl;
        volatile int never = 0;
        drain_ctl.abort = &never;
        for (int s = 0; s < STAGES1; ++s)
          if (issued[s]) wait_bounded(smem_u32(&full[s]), issued_phase[s], drain_ctl, 0);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
        const uint32_t b = it & 1u, aph = (it >> 1) & 1u;
        if (!wait_bounded(smem_u32(&tempty[b]), aph ^ 1u, ctl, 22) ||
            !wait_bounded(smem_u32(&full[stage]), phase, ctl, 23)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a_addr = smem_u32(stage_base + stage * STAGE1_BYTES);
        const uint64_t adesc = sw128_desc(a_addr, 16, 1024);
        const uint64_t bdesc =
            B_KMAJOR ? sw128_desc(a_addr + SLAB, 16, 1024) : sw128_desc(a_addr + SLAB, SLAB, 1024);
        constexpr uint32_t b_step = B_KMAJOR ? 2 : 256;  // 32 k: 32 bytes along a row, or 32 rows of 128 bytes
        constexpr uint32_t idesc = idesc_f8(128, BN1, B_KMAJOR);
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          umma_f8(tmem_base + b * BN1, adesc + (uint64_t)(2 * kk), bdesc + (uint64_t)(b_step * kk), idesc, kk > 0);
        umma_commit(smem_u32(&empty[stage]));
        if (!(gp.fault == 1 && it == 0)) umma_commit(smem_u32(&tfull[b]));
        if (++stage == STAGES1) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok && it > 0) {  // all issued MMAs must finish before the memory is freed
        Ctl drain_ctl = ctl;
        volatile int never = 0;
        drain_ctl.abort = &never;
        umma_commit(smem_u32(drain));
        wait_bounded(smem_u32(drain), 0, drain_ctl, 0);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q4 = warp & 3;  // tensor-memory lane quarter this warp may access
    const int row = q4 * 32 + lane;
    const int col0 = ((warp - 2) >> 2) * 64;
    const int m = min(tm * 128 + row, gp.M - 1);
    const float* sa = gp.SA + (long long)m * gp.KB;
    float* sbuf = scale_base + (warp - 2) * 128;
    const float* sb0;  // this lane's scales of B: columns lane, lane + 32 of the warp's 64 (or the tile's one)
    const float* sb1;
    if constexpr (TILE_B) {
      sb0 = gp.SB + (long long)tn * gp.sb_n;  // a tile's 128 columns are one block
      sb1 = sb0;
    } else {
      const int n = tn * BN1 + col0 + lane;
      sb0 = gp.SB + (long long)min(n, gp.N - 1) * gp.sb_n;
      sb1 = gp.SB + (long long)min(n + 32, gp.N - 1) * gp.sb_n;
    }
    float acc[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
    uint32_t it = 0;
    bool ok = true;
    for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
      const uint32_t b = it & 1u, aph = (it >> 1) & 1u;
      float s = __ldg(sa + kb);
      if constexpr (TILE_B) {
        s *= __ldg(sb0 + kb * gp.sb_k);
      } else {
        sbuf[b * 64 + lane] = __ldg(sb0 + kb * gp.sb_k);
        sbuf[b * 64 + 32 + lane] = __ldg(sb1 + kb * gp.sb_k);
      }
      ok = __all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&tfull[b]), aph, ctl, 24));
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q4 * 32) << 16) + b * BN1 + col0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        tmem_ld32(taddr + 32 * h, r);
        tmem_wait_ld();
        pin32(r);
        if (h == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&tempty[b]));
        }
        if constexpr (TILE_B) {
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[32 * h + i] = __fmaf_rn(__uint_as_float(r[i]), s, acc[32 * h + i]);
        } else {
          const float4* sv = reinterpret_cast<const float4*>(sbuf + b * 64 + 32 * h);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 v = sv[i];
            const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int e = 4 * i + j;
              acc[32 * h + e] = __fmaf_rn(__uint_as_float(r[e]), s * w[j], acc[32 * h + e]);
            }
          }
        }
      }
    }
    // the stages are idle once the last block's product is complete; the
    // partial tile takes their place
    if (ok) {
      float* part = reinterpret_cast<float*>(stage_base) + row * PART_LD + col0;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float4*>(part + 4 * i) =
            make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"((uint32_t)(2 * BN1)));
  }
  // rows rank, rank + S, ... of the tile: the slices' sums in rank order
  if (!*abort_flag) {
    const int rows = min(128, gp.M - tm * 128), cols = min(BN1, gp.N - tn * BN1);
    const uint32_t base = smem_u32(stage_base);
    for (int r = rank + S * warp; r < rows; r += S * (NUM_THREADS / 32)) {
      const long long out = (long long)(tm * 128 + r) * gp.ldc + (long long)tn * BN1;
      for (int c = lane; c < cols; c += 32) {
        const uint32_t at = base + (uint32_t)(r * PART_LD + c) * 4;
        float v;
        if (S == 1) {
          v = reinterpret_cast<const float*>(stage_base)[r * PART_LD + c];
        } else {
          v = ld_cluster(mapa_shared(at, 0));
          for (int k = 1; k < S; ++k) v += ld_cluster(mapa_shared(at, (uint32_t)k));
        }
        store_out(gp.C, out + c, gp.out_type, v);
      }
    }
  }
  allow_dependents();
  if (S > 1) cluster_sync();  // no CTA leaves while another reads its slice
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
bool make_map_2d(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t stride_bytes, uint32_t b0,
                 uint32_t b1) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {d0, d1};
  cuuint64_t strides[1] = {stride_bytes};
  cuuint32_t box[2] = {b0, b1};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using TileKernel = void (*)(const CUtensorMap, const CUtensorMap, const Params, int, DevPlan*);
constexpr TileKernel kTileKernels[2][2] = {{f8_gemm_tile_kernel<false, false>, f8_gemm_tile_kernel<false, true>},
                                           {f8_gemm_tile_kernel<true, false>, f8_gemm_tile_kernel<true, true>}};

struct F8Device {
  int sms = 0;
};
cudaError_t f8_device(int dev, F8Device& out) {
  static std::mutex mu;
  static F8Device devs[64];
  std::lock_guard<std::mutex> lock(mu);
  F8Device& d = devs[dev];
  if (!d.sms) {
    for (auto& row : kTileKernels)
      for (auto k : row) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM1_BYTES);
        if (e != cudaSuccess) return e;
      }
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (sms < 2) return cudaErrorInvalidDevice;
    d.sms = sms;
  }
  out = d;
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_f8_gemm(const F8GemmArgs& a, DevPlan* plan, cudaStream_t st, int fault,
                           unsigned long long wait_ns) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  F8Device fd;
  e = f8_device(dev, fd);
  if (e != cudaSuccess) return e;
  Params p;
  p.SA = a.SA;
  p.SB = a.SB;
  p.C = a.C;
  p.ldc = a.ldc;
  p.sb_n = a.sb_n;
  p.sb_k = a.sb_k;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.KB = (int)((a.K + BK - 1) / BK);
  p.mt = (int)((a.M + 127) / 128);
  p.nt = (int)((a.N + BN1 - 1) / BN1);
  p.out_type = a.out_type;
  const int es = a.out_type == RG_TYPE_F32 ? 4 : 2;
  p.vec_c = reinterpret_cast<uintptr_t>(a.C) % 16 == 0 && a.ldc * es % 16 == 0;
  p.fault = fault;
  p.wait_ns = wait_ns;
  CUtensorMap ma, mb;
  if (!make_map_2d(&ma, a.A, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.lda, BK, 128) ||
      !(a.b_kmajor ? make_map_2d(&mb, a.B, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.ldb, BK, 128)
                   : make_map_2d(&mb, a.B, (uint64_t)a.N, (uint64_t)a.K, (uint64_t)a.ldb, 128, BK)))
    return cudaErrorInvalidValue;
  const long long tiles = (long long)p.mt * p.nt;
  int S = 1;
  while (S < 8 && tiles * S * 2 <= fd.sms && p.KB >= 4 * S) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * S));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = SMEM1_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kTileKernels[a.b_kmajor][a.tile_b], ma, mb, p, S, plan);
}

}  // namespace rg
