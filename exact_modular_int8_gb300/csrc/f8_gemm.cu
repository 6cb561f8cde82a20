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
// Warp roles: warp 0 TMA producer, warps 1 (and 2, in the pair kernel) tensor
// memory and MMA issue, the rest of the first four copy the scales to shared
// memory, warps 4..11 epilogue.  Every wait is bounded as in the residue
// product.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "f8_kernels.h"
#include "rg_kernels.h"
#include "rg_tc.cuh"

namespace rg {
namespace {

constexpr int BK = 128;  // values of k per block and pipeline stage: one 128-byte swizzle row
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 128 + 32 * EPI_WARPS;
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
  int keep_status;
  unsigned long long wait_ns;
};

__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// The call's status, in place of a memset before the kernel: by the grid's first
// thread as it starts, a time limit (which no wait can have used up yet) before
// any CTA could write to it.
__device__ __forceinline__ void clear_status(const Params& gp, DevPlan* plan) {
  if (blockIdx.x == 0 && !gp.keep_status) {
    plan->status = 0;
    plan->timeout_where = 0;
  }
}

// One thread of a converged warp.  The issuing warps run their loops whole and
// elect a thread for the MMAs alone: their descriptors then stay in uniform
// registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// Waits for a phase of both barriers; by whole warps (the answer is the same for all lanes).
__device__ __forceinline__ bool wait_both(uint32_t bar0, uint32_t par0, uint32_t bar1, uint32_t par1, const Ctl& ctl,
                                          int where) {
  const bool r0 = mbar_try_wait(bar0, par0), r1 = mbar_try_wait(bar1, par1);  // the two round trips overlap
  bool ok = true;
  if (!r0) ok = wait_bounded(bar0, par0, ctl, where);
  if (!r1 && ok) ok = wait_bounded(bar1, par1, ctl, where + 1);
  return __all_sync(0xFFFFFFFFu, ok);
}

// Shared-memory matrix descriptor, 64-byte swizzle.  lbo/sbo in bytes.
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (sw128_desc(saddr, lbo, sbo) & ~((uint64_t)7 << 61)) | (uint64_t)4 << 61;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// ---------------------------------------------------------------------------
// Scales.  One or two warps copy the CTA's scales to shared memory, KC blocks of 128
// at a time and two such chunks deep, so that the epilogue reads them there:
// sa[KC][128 rows], sb[KC][NC columns] (or one value per 128 columns).  The
// scales lie with the blocks of a row next to each other (or B's columns, for
// an untransposed B), so a warp's copy instruction covers a few short runs of
// consecutive words; loading them a row to a lane in the epilogue itself took
// three times as long as all its other work.
// ---------------------------------------------------------------------------
constexpr int KC = 8;
constexpr int SCALE_BUFS = 2;
template <int NC>
struct ScaleChunk {
  float a[KC][128 + 4];  // rows padded: the copies of one instruction fall into different banks
  float b[KC][NC + 4];
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrive on the barrier once this thread's copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Blocks kb0 .. kb0 + KC - 1 (at most kb_end) of rows [m0, m0 + 128) and columns
// [n0, n0 + NC), by NT threads t.  Entries past the matrix repeat its last.
template <int NC, bool TILE_B, int NT>
__device__ __forceinline__ void load_scales(const Params& gp, ScaleChunk<NC>& c, int m0, int n0, int kb0, int kb_end,
                                            int t) {
  const int kbi = t & (KC - 1), kb = min(kb0 + kbi, kb_end - 1);
#pragma unroll 4
  for (int r = t >> 3; r < 128; r += NT / 8)
    cp_async4(smem_u32(&c.a[kbi][r]), gp.SA + (long long)min(m0 + r, gp.M - 1) * gp.KB + kb);
  if constexpr (TILE_B) {
    if (t < KC * (NC / 128)) {
      const int h = t >> 3;
      cp_async4(smem_u32(&c.b[kbi][h]),
                gp.SB + (long long)min(n0 / 128 + h, (gp.N - 1) / 128) * gp.sb_n + kb * gp.sb_k);
    }
  } else if (gp.sb_k == 1) {
#pragma unroll 4
    for (int n = t >> 3; n < NC; n += NT / 8)
      cp_async4(smem_u32(&c.b[kbi][n]), gp.SB + (long long)min(n0 + n, gp.N - 1) * gp.sb_n + kb);
  } else {
    for (int q = 0; q < KC; ++q)
      for (int n = t; n < NC; n += NT)
        cp_async4(smem_u32(&c.b[q][n]),
                  gp.SB + (long long)min(n0 + n, gp.N - 1) * gp.sb_n + (long long)min(kb0 + q, kb_end - 1) * gp.sb_k);
  }
}

__device__ __forceinline__ void store_out(void* C, long long at, int type, float v) {
  if (type == RG_TYPE_F32) static_cast<float*>(C)[at] = v;
  else if (type == RG_TYPE_F16) static_cast<__half*>(C)[at] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(C)[at] = __float2bfloat16_rn(v);
}

// Pairs of fp32 (fma.rn.f32x2: two multiply-adds per instruction).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ uint64_t pack2u(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrive on a barrier of another CTA of the cluster without releasing memory:
// it only reports tensor-memory reads, ordered by the tcgen05 fence before it.
// (A release at cluster scope drains the warp's memory operations; it took 1100
// of the 2500 cycles that a 128-block then cost.)
__device__ __forceinline__ void mbar_arrive_relaxed_cluster(uint32_t bar_cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster_addr) : "memory");
}

// One epilogue warp's fp32 sums of 32 rows x COLS columns, in pairs of columns,
// and how a block's product is added to them.  `release` runs once the last read
// of tensor memory is complete; 64 columns are read at a time, so that it runs
// before most of the arithmetic.
//
// With one scale for all the columns (TILE_B) a lane holds a row: acc += p s, the
// column scale already in s.  (8192 x 8192 x 4096, at this choice: 239 us, 284 in the
// other form.)
template <int COLS, bool TILE_B>
struct Sums {
  static constexpr int kRows = 1;
  uint64_t acc[1][COLS / 2];
  static __device__ __forceinline__ int row(int lane, int) { return lane; }
  static __device__ __forceinline__ int col(int, int j) { return 2 * j; }

  template <typename F>
  __device__ __forceinline__ void add(uint32_t taddr, const float (&s)[1], const float*, F&& release) {
    const uint64_t s2 = pack2(s[0], s[0]);
#pragma unroll
    for (int h = 0; h < COLS / 64; ++h) {
      uint32_t c[32], d[32];
      tmem_ld32(taddr + 64 * h, c);
      tmem_ld32(taddr + 64 * h + 32, d);
      tmem_wait_ld();
      pin32(c);
      pin32(d);
      if (h == COLS / 64 - 1) release();
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[0][32 * h + i] = fma2(pack2u(c[2 * i], c[2 * i + 1]), s2, acc[0][32 * h + i]);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        acc[0][32 * h + 16 + i] = fma2(pack2u(d[2 * i], d[2 * i + 1]), s2, acc[0][32 * h + 16 + i]);
    }
  }
};
// With a scale for each column: acc += (p s[row]) sb[column], in the shape of an MMA
// fragment.  Registers 4 j + {0, 1} of a read of 16 rows are row lane / 4, columns
// 8 j + 2 (lane & 3) + {0, 1}, registers 4 j + {2, 3} the same of row lane / 4 + 8, so
// a lane needs the scales of a quarter of the columns.  With a row to a lane it
// needs all of them: 32 loads of 16 bytes per block and warp, each filling 512
// bytes of registers, were a third of the time.  The read of 32 columns is under way
// during the arithmetic on the 32 before.  (8192 x 8192 x 4096: 365 us, 382 with 64
// columns read at a time and then added, 425 with a row to a lane.  The other form,
// with half the arithmetic, gains nothing from smaller reads: 239 us against 236.)
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : RG_R8(0), RG_R8(8)
      : "r"(taddr));
}
template <int COLS>
struct Sums<COLS, false> {
  static constexpr int kRows = 4;
  uint64_t acc[4][COLS / 8];
  static __device__ __forceinline__ int row(int lane, int i) { return (lane >> 2) + 8 * i; }
  static __device__ __forceinline__ int col(int lane, int j) { return 8 * j + 2 * (lane & 3); }

  template <typename F>
  __device__ __forceinline__ void add(uint32_t taddr, const float (&s)[4], const float* sb, F&& release) {
    const uint64_t s2[4] = {pack2(s[0], s[0]), pack2(s[1], s[1]), pack2(s[2], s[2]), pack2(s[3], s[3])};
    const int t4 = threadIdx.x & 3;
    uint32_t c[2][2][16];  // by chunk of 32 columns: rows 0..15 and 16..31
    tmem_ld_frag(taddr, c[0][0]);
    tmem_ld_frag(taddr + (16u << 16), c[0][1]);
#pragma unroll
    for (int h = 0; h < COLS / 32; ++h) {
      const int b = h & 1;
      uint64_t w[4];
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(c[b][i >> 4][i & 15]));
      if (h + 1 < COLS / 32) {
        tmem_ld_frag(taddr + 32 * (h + 1), c[b ^ 1][0]);
        tmem_ld_frag(taddr + 32 * (h + 1) + (16u << 16), c[b ^ 1][1]);
      } else {
        release();
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint64_t*>(sb + 32 * h + 8 * j + 2 * t4);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint64_t& a = acc[2 * q + i][4 * h + j];
            a = fma2(mul2(pack2u(c[b][q][4 * j + 2 * i], c[b][q][4 * j + 2 * i + 1]), s2[2 * q + i]), w[j], a);
          }
    }
  }
};

// ---------------------------------------------------------------------------
// Tiles of 128 x 128, one per cluster of S CTAs: each CTA sums a slice of K,
// and the slices are joined through distributed shared memory in rank order.
// For products that one wave of CTAs holds, where the time is the latency of
// set-up, K / S / 128 blocks of 0.3 us and the join: 512 x 4096 x 4096 12.7 us,
// 128 x 4096 x 4096 (S = 4) 7.9 us, 1000 x 1544 x 2056 10.1 us, one after another
// with operands in L2 (13.8, 8.2 and 10.7 with a row of the join at a time); with
// operands from memory 13.4, 9.2 and 10.2.
// ---------------------------------------------------------------------------
constexpr int BN1 = 128;
constexpr int STAGES1 = 6;
constexpr int STAGE1_BYTES = 2 * SLAB;
constexpr int PART_LD = BN1 + 4;  // floats per row of a CTA's partial tile, kept where the stages were
static_assert(128 * PART_LD * 4 <= STAGES1 * STAGE1_BYTES, "partial tile");
constexpr int SCALE1_BYTES = SCALE_BUFS * (int)sizeof(ScaleChunk<BN1>);
constexpr int SMEM1_BYTES = 1024 + STAGES1 * STAGE1_BYTES + SCALE1_BYTES + 256;
static_assert(SMEM1_BYTES <= 232448, "shared memory");

// Four neighbouring entries of C's row from column c of the tile on.
__device__ __forceinline__ void store4(const Params& gp, long long out, int c, int cols, float4 v) {
  if (gp.vec_c && c + 4 <= cols) {
    if (gp.out_type == RG_TYPE_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(gp.C) + out) = v;
    } else {
      uint2 w;
      if (gp.out_type == RG_TYPE_F16) {
        const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
        w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(gp.C) + out) = w;
    }
  } else {
    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < cols) store_out(gp.C, out + q, gp.out_type, e[q]);
  }
}

// Rows rank, rank + S, ... of the tile: the slices' sums in rank order.  A warp
// fetches all of its rows (S = 1: half of them) from every slice before it adds
// the first, so that the way to another CTA's shared memory, most of a
// microsecond, is waited for once.  The CTAs part when their reads are done,
// before their stores to C.
template <int S>
__device__ __forceinline__ void join_slices(const Params& gp, uint32_t part, int rank, int tm, int tn, int warp, int lane,
                                            bool live) {
  constexpr int WARPS = NUM_THREADS / 32, ROWS = (128 / S + WARPS - 1) / WARPS, R = S == 1 ? (ROWS + 1) / 2 : ROWS;
  const int rows = min(128, gp.M - tm * 128), cols = min(BN1, gp.N - tn * BN1);
  const int c = 4 * lane;  // this lane's columns
#pragma unroll
  for (int i0 = 0; i0 < ROWS; i0 += R) {
    float4 v[S][R];
#pragma unroll
    for (int k = 0; k < S; ++k)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = rank + S * (warp + WARPS * (i0 + i));
        v[k][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (live && r < rows && c < cols) {
          const uint32_t at = part + (uint32_t)(r * PART_LD + c) * 4;
          v[k][i] = ld_cluster4(S == 1 ? at : mapa_shared(at, (uint32_t)k));
        }
      }
#pragma unroll
    for (int k = 1; k < S; ++k)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        v[0][i].x += v[k][i].x;
        v[0][i].y += v[k][i].y;
        v[0][i].z += v[k][i].z;
        v[0][i].w += v[k][i].w;
      }
    __syncwarp();
    if (S > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = rank + S * (warp + WARPS * (i0 + i));
      if (live && r < rows && c < cols)
        store4(gp, (long long)(tm * 128 + r) * gp.ldc + (long long)tn * BN1 + c, c, cols, v[0][i]);
    }
  }
  __syncwarp();
  if (S > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <bool B_KMAJOR, bool TILE_B>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    f8_gemm_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ Params gp, int S, DevPlan* plan) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stage_base = smem;
  ScaleChunk<BN1>* scales = reinterpret_cast<ScaleChunk<BN1>*>(smem + STAGES1 * STAGE1_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES1 * STAGE1_BYTES + SCALE1_BYTES);
  uint64_t* full = bars;
  uint64_t* done = bars + STAGES1;        // the stage's MMAs are complete
  uint64_t* tempty = bars + 2 * STAGES1;  // by accumulator
  uint64_t* sfull = tempty + 2;
  uint64_t* sempty = sfull + SCALE_BUFS;
  uint64_t* drain = sempty + SCALE_BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
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
      mbar_init(smem_u32(&done[s]), 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&tempty[b]), EPI_WARPS);
    for (int b = 0; b < SCALE_BUFS; ++b) {
      mbar_init(smem_u32(&sfull[b]), 64);
      mbar_init(smem_u32(&sempty[b]), EPI_WARPS);
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
  // the set-up above overlaps the predecessor's tail
  wait_for_predecessor();
  allow_dependents();
  if (threadIdx.x == 0) clear_status(gp, plan);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool issued[STAGES1] = {};
      uint32_t issued_phase[STAGES1] = {};
      bool ok = true;
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        if (!wait_bounded(smem_u32(&done[stage]), phase ^ 1u, ctl, 21)) {
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
    const uint32_t a_addr = smem_u32(stage_base), b_addr = a_addr + SLAB;
    const uint64_t adesc0 = sw128_desc(a_addr, 16, 1024);
    const uint64_t bdesc0 = B_KMAJOR ? sw128_desc(b_addr, 16, 1024) : sw128_desc(b_addr, SLAB, 1024);
    constexpr uint32_t b_step = B_KMAJOR ? 2 : 256;  // 32 k: 32 bytes along a row, or 32 rows of 128 bytes
    constexpr uint32_t idesc = idesc_f8(128, BN1, B_KMAJOR);
    int stage = 0;
    uint32_t phase = 0, it = 0;
    bool ok = true;
    for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
      const uint32_t b = it & 1u, aph = (it >> 1) & 1u;
      ok = wait_both(smem_u32(&tempty[b]), aph ^ 1u, smem_u32(&full[stage]), phase, ctl, 22);
      if (!ok) break;
      tc_fence_after();
      const uint64_t off = (uint64_t)(stage * (STAGE1_BYTES >> 4));
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          umma_f8(tmem_base + b * BN1, adesc0 + off + (uint64_t)(2 * kk), bdesc0 + off + (uint64_t)(b_step * kk), idesc,
                  kk > 0);
        if (!(gp.fault == 1 && it == 0)) umma_commit(smem_u32(&done[stage]));
      }
      __syncwarp();
      if (++stage == STAGES1) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok && it > 0) {  // all issued MMAs must finish before the memory is freed
      Ctl drain_ctl = ctl;
      volatile int never = 0;
      drain_ctl.abort = &never;
      if (elect_one()) umma_commit(smem_u32(drain));
      __syncwarp();
      wait_bounded(smem_u32(drain), 0, drain_ctl, 0);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ scales
    int c = 0;
    for (int kb = kb_lo; kb < kb_hi; kb += KC, ++c) {
      const int b = c & 1;
      if (!wait_bounded(smem_u32(&sempty[b]), ((c >> 1) & 1u) ^ 1u, ctl, 25)) break;
      load_scales<BN1, TILE_B, 64>(gp, scales[b], tm * 128, tn * BN1, kb, kb_hi, threadIdx.x - 64);
      cp_async_arrive(smem_u32(&sfull[b]));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------------------------------------ epilogue
    const int q4 = warp & 3;  // tensor-memory lane quarter this warp may access
    constexpr int WC = BN1 * 4 / EPI_WARPS;  // columns per warp
    const int col0 = ((warp - 4) >> 2) * WC;
    using Acc = Sums<WC, TILE_B>;
    Acc sums = {};
    uint32_t it = 0, phase = 0;
    int st = 0;  // pipeline stage
    bool ok = true;
    for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
      const uint32_t b = it & 1u;
      const int c = (int)it / KC, kbi = (int)it % KC;
      const ScaleChunk<BN1>& sc = scales[c & 1];
      ok = kbi != 0 || wait_bounded(smem_u32(&sfull[c & 1]), (c >> 1) & 1u, ctl, 26);
      ok = __all_sync(0xFFFFFFFFu, ok && wait_bounded(smem_u32(&done[st]), phase, ctl, 24));
      if (++st == STAGES1) {
        st = 0;
        phase ^= 1u;
      }
      if (!ok) break;
      tc_fence_after();
      float s[Acc::kRows];
#pragma unroll
      for (int i = 0; i < Acc::kRows; ++i) {
        s[i] = sc.a[kbi][q4 * 32 + Acc::row(lane, i)];
        if constexpr (TILE_B) s[i] *= sc.b[kbi][0];
      }
      sums.add(tmem_base + ((uint32_t)(q4 * 32) << 16) + b * BN1 + col0, s, &sc.b[kbi][col0], [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(smem_u32(&tempty[b]));
      });
      if (kbi == KC - 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sempty[c & 1]));
      }
    }
    // the stages are idle once the last block's product is complete; the
    // partial tile takes their place
    if (ok) {
      float* part = reinterpret_cast<float*>(stage_base) + q4 * 32 * PART_LD + col0;
      if constexpr (TILE_B) {  // 16 bytes at a time
#pragma unroll
        for (int j = 0; j < WC / 2; j += 2)
          *reinterpret_cast<ulonglong2*>(part + lane * PART_LD + 2 * j) =
              make_ulonglong2(sums.acc[0][j], sums.acc[0][j + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < Acc::kRows; ++i)
#pragma unroll
          for (int j = 0; j < WC / 8; ++j)
            *reinterpret_cast<uint64_t*>(part + Acc::row(lane, i) * PART_LD + Acc::col(lane, j)) = sums.acc[i][j];
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  if (S > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"((uint32_t)(2 * BN1)));
  }
  const bool live = !*abort_flag;
  const uint32_t part = smem_u32(stage_base);
  if (S == 1) join_slices<1>(gp, part, rank, tm, tn, warp, lane, live);
  else if (S == 2) join_slices<2>(gp, part, rank, tm, tn, warp, lane, live);
  else if (S == 4) join_slices<4>(gp, part, rank, tm, tn, warp, lane, live);
  else join_slices<8>(gp, part, rank, tm, tn, warp, lane, live);
}

// ---------------------------------------------------------------------------
// Tiles of 256 x 256 on CTA pairs (cta_group::2), persistent.  Each CTA holds
// 128 rows of A and 128 columns of B per stage and receives its own 128 rows
// of the accumulator; its eight epilogue warps each keep 32 rows x 128 columns
// of fp32 sums in registers (128 of them a lane).
//
// The tile's two column halves are separate MMAs (M = 256, N = 128, each CTA
// holding 64 of the 128 columns), issued by a warp each, into two alternating
// accumulators of their own.  A block's product, its read-back and the way back
// through the barriers is a chain of about 1300 cycles with whole 256-column
// MMAs, of which only two are in flight; the halves' chains are shorter and
// interleave.
//
// 8192 x 8192 x 4096: 236 us, 2330 TFLOP/s, half of the E4M3 instruction rate (the
// tensor pipe is active 46% of the time).  A block of a tile takes 1050 cycles
// where its MMAs take 512 and the same loop with an empty epilogue 720: an
// epilogue warp waits for 165, has read its columns 440 later and needs the rest
// for the multiply-adds and a share of the stores, with two warps to a scheduler.
// More epilogue warps (16: spills, 293 us), 256 x 192 tiles with twelve warps (271
// us) and single-CTA 128 x 192 tiles (261 us) were slower; one 256-column MMA for
// both halves took the same time.  With a scale for each of B's rows: 366 us, 1535
// cycles a block (380 us with fp32 results); 2048 x 4096 x 8100 108 us.
//
// The block is launched with 168 registers a thread; the first warpgroup
// (producer, MMA issue, scales) gives up 112 of them and the two epilogue
// warpgroups take 56 more each: 56 + 2 * 224 = 3 * 168.
// ---------------------------------------------------------------------------
constexpr int BN2 = 256;
constexpr int STAGES2 = 5;
constexpr int STAGE2_BYTES = 2 * SLAB;
constexpr int HALF_SLAB = SLAB / 2;  // a CTA's 64 columns of one half
constexpr int PAIR_COLS = BN2 * 4 / EPI_WARPS;  // columns per epilogue warp
constexpr int OUT_BUF = 32 * 64;  // 64 bytes of each of a warp's rows
constexpr int OUT_WARP = 2 * OUT_BUF;
constexpr int SCALE2_BYTES = SCALE_BUFS * (int)sizeof(ScaleChunk<BN2>);
constexpr int SMEM2_BYTES = 1024 + STAGES2 * STAGE2_BYTES + EPI_WARPS * OUT_WARP + SCALE2_BYTES + 256;
static_assert(SMEM2_BYTES <= 232448, "shared memory");

__device__ __forceinline__ void umma_f8_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster_addr,
                                                 int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(c0), "r"(c1)
      : "memory");
}

// This warp's 32 rows x 128 columns of sums to C, 64 bytes of each row at a time
// through two alternating staging buffers (16-byte chunks swizzled as the TMA's
// 64-byte mode has them).  Where C's rows start on 16-byte boundaries a TMA
// store takes each buffer away and cuts it to the matrix; else the warp writes
// it entry by entry.
template <int ES>  // bytes per entry of C
__device__ __forceinline__ void stage_pair(uint8_t* dst, float2 f, int type) {
  if constexpr (ES == 4) *reinterpret_cast<float2*>(dst) = f;
  else if (type == RG_TYPE_F16) *reinterpret_cast<__half2*>(dst) = __floats2half2_rn(f.x, f.y);
  else *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(f.x, f.y);
}
template <int ES>
__device__ __forceinline__ uint32_t packed(float2 f, int type) {
  uint32_t w;
  stage_pair<ES>(reinterpret_cast<uint8_t*>(&w), f, type);
  return w;
}
template <int ES, bool TILE_B>
__device__ __forceinline__ void store_rows(const Params& gp, const CUtensorMap* tmC,
                                           const Sums<PAIR_COLS, TILE_B>& sums, uint8_t* stage, int row0, int col0,
                                           int lane) {
  constexpr int COLS = 64 / ES;
  const int rows = min(32, gp.M - row0);
#pragma unroll
  for (int c = 0; c < PAIR_COLS / COLS; ++c) {
    uint8_t* buf = stage + (c & 1) * OUT_BUF;
    if (gp.vec_c) {  // the store that used this buffer before has read it
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();
    }
    if constexpr (TILE_B) {  // a row to a lane: 16 bytes at a time
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 w;
        if constexpr (ES == 4) {
          const float2 f = unpack2(sums.acc[0][c * (COLS / 2) + 2 * i]);
          const float2 h = unpack2(sums.acc[0][c * (COLS / 2) + 2 * i + 1]);
          w = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(h.x), __float_as_uint(h.y));
        } else {
          uint32_t p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = packed<ES>(unpack2(sums.acc[0][c * (COLS / 2) + 4 * i + j]), gp.out_type);
          w = make_uint4(p[0], p[1], p[2], p[3]);
        }
        *reinterpret_cast<uint4*>(buf + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (lane >> 2) + 8 * i;
#pragma unroll
        for (int j = 0; j < COLS / 8; ++j) {
          const int at = (8 * j + 2 * (lane & 3)) * ES;  // byte within the row's 64
          stage_pair<ES>(buf + r * 64 + (((at >> 4) ^ ((r >> 1) & 3)) << 4) + (at & 15),
                         unpack2(sums.acc[i][c * (COLS / 8) + j]), gp.out_type);
        }
      }
    }
    const int cc = col0 + c * COLS;
    if (gp.vec_c) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (cc < gp.N)
          asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                           reinterpret_cast<uint64_t>(tmC)),
                       "r"(smem_u32(buf)), "r"(cc), "r"(row0)
                       : "memory");
        bulk_commit();
      }
    } else {
      __syncwarp();
      const int cols = min(COLS, gp.N - cc);
      uint8_t* out = static_cast<uint8_t*>(gp.C) + ((long long)row0 * gp.ldc + cc) * ES;
      for (int r = 0; r < rows; ++r)
        for (int j = lane; j < cols; j += 32) {
          const int at = j * ES;
          const uint8_t* src = buf + r * 64 + (((at >> 4) ^ ((r >> 1) & 3)) << 4) + (at & 15);
          if constexpr (ES == 4)
            reinterpret_cast<uint32_t*>(out + (long long)r * gp.ldc * ES)[j] = *reinterpret_cast<const uint32_t*>(src);
          else
            reinterpret_cast<uint16_t*>(out + (long long)r * gp.ldc * ES)[j] = *reinterpret_cast<const uint16_t*>(src);
        }
      __syncwarp();
    }
  }
}

template <bool B_KMAJOR, bool TILE_B>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    f8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmC, const __grid_constant__ Params gp, DevPlan* plan) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t rank = cluster_rank();
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stage_base = smem;
  uint8_t* out_base = smem + STAGES2 * STAGE2_BYTES;
  ScaleChunk<BN2>* scales = reinterpret_cast<ScaleChunk<BN2>*>(out_base + EPI_WARPS * OUT_WARP);
  uint64_t* bars = reinterpret_cast<uint64_t*>(out_base + EPI_WARPS * OUT_WARP + SCALE2_BYTES);
  uint64_t* full = bars;
  uint64_t* done = bars + STAGES2;         // by half * STAGES2 + stage: the half's MMAs of the stage are complete
  uint64_t* tempty = bars + 3 * STAGES2;  // by half * 2 + accumulator
  uint64_t* sfull = tempty + 4;
  uint64_t* sempty = sfull + SCALE_BUFS;
  uint64_t* drain = sempty + SCALE_BUFS;  // by half
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ctl ctl{abort_flag, &plan->status, &plan->timeout_where, gp.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES2; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&done[s]), 1);
      mbar_init(smem_u32(&done[STAGES2 + s]), 1);
    }
    for (int b = 0; b < 4; ++b) mbar_init(smem_u32(&tempty[b]), EPI_WARPS);  // the half's warps of both CTAs
    for (int b = 0; b < SCALE_BUFS; ++b) {
      mbar_init(smem_u32(&sfull[b]), 32);
      mbar_init(smem_u32(&sempty[b]), EPI_WARPS);
    }
    for (int h = 0; h < 2; ++h) mbar_init(smem_u32(&drain[h]), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {  // one warp in each CTA allocates for the pair
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"((uint32_t)(2 * BN2)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  __syncwarp();  // the cluster's barrier is for whole warps
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // the set-up above overlaps the predecessor's tail
  wait_for_predecessor();
  allow_dependents();
  if (threadIdx.x == 0) clear_status(gp, plan);
  const int total = gp.mt * gp.nt;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = cid; t < total && ok; t += ncl) {
        const int tn = t / gp.mt, tm = t - tn * gp.mt;
        for (int kb = 0; kb < gp.KB; ++kb) {
          if (!wait_bounded(smem_u32(&done[stage]), phase ^ 1u, ctl, 31) ||
              !wait_bounded(smem_u32(&done[STAGES2 + stage]), phase ^ 1u, ctl, 31)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = smem_u32(&full[stage]);
          if (rank == 0) mbar_arrive_expect_tx(fb_local, 2 * STAGE2_BYTES);
          const uint32_t fb = mapa_shared(fb_local, 0);
          const uint32_t a_dst = smem_u32(stage_base + stage * STAGE2_BYTES);
          tma_load_2d_pair(a_dst, &tmA, fb, kb * BK, tm * 256 + (int)rank * 128);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t b_dst = a_dst + SLAB + h * HALF_SLAB;
            const int n0 = tn * BN2 + h * 128 + (int)rank * 64;
            if constexpr (B_KMAJOR) tma_load_2d_pair(b_dst, &tmB, fb, kb * BK, n0);
            else tma_load_2d_pair(b_dst, &tmB, fb, n0, kb * BK);
          }
          if (++stage == STAGES2) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    if ((warp == 1 || warp == 2) && rank == 0) {
      // ---------------------------------------------------------- MMA issuers (first CTA), one warp per half
      const int half = __shfl_sync(0xFFFFFFFFu, warp - 1, 0);
      const uint32_t a_addr = smem_u32(stage_base), b_addr = a_addr + SLAB + half * HALF_SLAB;
      const uint64_t adesc0 = sw128_desc(a_addr, 16, 1024);
      // N-major: 64 columns are one 64-byte swizzle row per k, eight k to a group of 512 bytes
      const uint64_t bdesc0 = B_KMAJOR ? sw128_desc(b_addr, 16, 1024) : sw64_desc(b_addr, HALF_SLAB, 512);
      constexpr uint32_t b_step = B_KMAJOR ? 2 : 128;  // 32 k: 32 bytes along a row, or 32 rows of 64 bytes
      constexpr uint32_t idesc = idesc_f8(256, 128, B_KMAJOR);
      int stage = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int t = cid; t < total && ok; t += ncl) {
        for (int kb = 0; kb < gp.KB; ++kb, ++it) {
          const uint32_t b = it & 1u, aph = (it >> 1) & 1u;
          ok = wait_both(smem_u32(&tempty[half * 2 + b]), aph ^ 1u, smem_u32(&full[stage]), phase, ctl, 32);
          if (!ok) break;
          tc_fence_after();
          const uint64_t off = (uint64_t)(stage * (STAGE2_BYTES >> 4));
          const uint32_t d = tmem_base + (half * 2 + b) * 128;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)
              umma_f8_pair(d, adesc0 + off + (uint64_t)(2 * kk), bdesc0 + off + (uint64_t)(b_step * kk), idesc, kk > 0);
            if (!(gp.fault == 1 && it == 0)) umma_commit_pair(smem_u32(&done[half * STAGES2 + stage]));
          }
          __syncwarp();
          if (++stage == STAGES2) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && it > 0) {  // all issued MMAs must finish before the memory is freed
        Ctl drain_ctl = ctl;
        volatile int never = 0;
        drain_ctl.abort = &never;
        if (elect_one()) umma_commit_pair_local(smem_u32(&drain[half]));
        __syncwarp();
        wait_bounded(smem_u32(&drain[half]), 0, drain_ctl, 0);
      }
    }
    if (warp == 3) {
      // ---------------------------------------------------------- scales (both CTAs)
      int c = 0;
      bool ok = true;
      for (int t = cid; t < total && ok; t += ncl) {
        const int tn = t / gp.mt, tm = t - tn * gp.mt;
        for (int kb = 0; kb < gp.KB && ok; kb += KC, ++c) {
          const int b = c & 1;
          ok = wait_bounded(smem_u32(&sempty[b]), ((c >> 1) & 1u) ^ 1u, ctl, 35);
          if (!ok) break;
          load_scales<BN2, TILE_B, 32>(gp, scales[b], tm * 256 + (int)rank * 128, tn * BN2, kb, gp.KB, lane);
          cp_async_arrive(smem_u32(&sfull[b]));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int q4 = warp & 3, ew = warp - 4;
    const int half = ew / (EPI_WARPS / 2);
    const int col = (ew >> 2) * PAIR_COLS;  // of the tile
    uint8_t* stage = out_base + ew * OUT_WARP;
    const uint32_t tempty_leader[2] = {mapa_shared(smem_u32(&tempty[half * 2]), 0),
                                       mapa_shared(smem_u32(&tempty[half * 2 + 1]), 0)};
    const uint32_t lane_addr = tmem_base + ((uint32_t)(q4 * 32) << 16) + half * 256 + (col & 127);
    uint32_t it = 0, phase = 0;
    int chunk = 0, st = 0;  // pipeline stage
    bool ok = true;
    for (int t = cid; t < total && ok; t += ncl) {
      const int tn = t / gp.mt, tm = t - tn * gp.mt;
      const int row0 = tm * 256 + (int)rank * 128 + q4 * 32, col0 = tn * BN2 + col;
      using Acc = Sums<PAIR_COLS, TILE_B>;
      Acc sums = {};
      for (int kb = 0; kb < gp.KB; ++kb, ++it) {
        const uint32_t b = it & 1u;
        const int kbi = kb % KC;
        const ScaleChunk<BN2>& sc = scales[chunk & 1];
        ok = kbi != 0 || wait_bounded(smem_u32(&sfull[chunk & 1]), (chunk >> 1) & 1u, ctl, 36);
        ok = __all_sync(0xFFFFFFFFu, ok && wait_bounded(smem_u32(&done[half * STAGES2 + st]), phase, ctl, 34));
        if (++st == STAGES2) {
          st = 0;
          phase ^= 1u;
        }
        if (!ok) break;
        tc_fence_after();
        float s[Acc::kRows];
#pragma unroll
        for (int i = 0; i < Acc::kRows; ++i) {
          s[i] = sc.a[kbi][q4 * 32 + Acc::row(lane, i)];
          if constexpr (TILE_B) s[i] *= sc.b[kbi][half];
        }
        sums.add(lane_addr + b * 128, s, &sc.b[kbi][col], [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed_cluster(tempty_leader[b]);
        });
        if (kbi == KC - 1 || kb == gp.KB - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sempty[chunk & 1]));
          ++chunk;
        }
      }
      if (ok && row0 < gp.M && col0 < gp.N) {
        if (gp.out_type == RG_TYPE_F32) store_rows<4, TILE_B>(gp, &tmC, sums, stage, row0, col0, lane);
        else store_rows<2, TILE_B>(gp, &tmC, sums, stage, row0, col0, lane);
      }
    }
    bulk_wait0();
  }

  __syncwarp();  // whole warps again before the abort check and the barriers below
  if (*abort_flag) {
    // an aborted role may leave copies in flight that signal either CTA:
    // give them time to land before the pair leaves
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA frees the pair's memory while the other still uses it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"((uint32_t)(2 * BN2)));
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// The encoder is a driver function: it needs a current context, which a host
// thread has only after a runtime call that makes one, and a product in a new
// thread comes here before any other.  It is made where the encoder has failed
// (the other calls pay nothing).
bool make_map_2d(CUtensorMap* m, int dev, const void* base, uint64_t d0, uint64_t d1, uint64_t stride_bytes, uint32_t b0,
                 uint32_t b1, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B,
                 CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {d0, d1};
  cuuint64_t strides[1] = {stride_bytes};
  cuuint32_t box[2] = {b0, b1};
  cuuint32_t es[2] = {1, 1};
  auto encode = [&] {
    return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return encode() || (cudaSetDevice(dev) == cudaSuccess && encode());
}

cudaLaunchConfig_t cluster_config(dim3 grid, int threads, int smem, cudaStream_t st, int cluster, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

using TileKernel = void (*)(const CUtensorMap, const CUtensorMap, const Params, int, DevPlan*);
constexpr TileKernel kTileKernels[2][2] = {{f8_gemm_tile_kernel<false, false>, f8_gemm_tile_kernel<false, true>},
                                           {f8_gemm_tile_kernel<true, false>, f8_gemm_tile_kernel<true, true>}};

using PairKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const Params, DevPlan*);
constexpr PairKernel kPairKernels[2][2] = {{f8_gemm_pair_kernel<false, false>, f8_gemm_pair_kernel<false, true>},
                                           {f8_gemm_pair_kernel<true, false>, f8_gemm_pair_kernel<true, true>}};

struct F8Device {
  int sms = 0, max_pairs = 0;
  int max_slices[4] = {};  // clusters of 1, 2, 4, 8 CTAs of the one-wave kernel that are resident together
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
    for (auto& row : kPairKernels)
      for (auto k : row) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM2_BYTES);
        if (e != cudaSuccess) return e;
      }
    // not every SM can be paired, or put into a larger cluster, within its GPC
    cudaLaunchAttribute attr[2];
    auto resident = [&](const void* kernel, int smem, int cluster) {
      const int ctas = sms / cluster * cluster;
      cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)ctas), NUM_THREADS, smem, nullptr, cluster, attr);
      int n = 0;
      if (ctas == 0) return 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();  // the query's own failure is not the call's
        n = sms / cluster;
      }
      return n;
    };
    d.max_pairs = resident(reinterpret_cast<const void*>(kPairKernels[1][1]), SMEM2_BYTES, 2);
    d.max_slices[0] = sms;
    for (int i = 1; i < 4; ++i)
      d.max_slices[i] = resident(reinterpret_cast<const void*>(kTileKernels[1][1]), SMEM1_BYTES, 1 << i);
    d.sms = sms;
  }
  out = d;
  return cudaSuccess;
}

// Where the warp-level kernel, whose warps split K but whose blocks do not, is
// faster than padded tiles, which do.  One launch after another, us, the
// warp-level kernel first; rows x columns x K:
//   to 8 rows     at nearly every size (8 x 1024 x 4096 3.5 / 4.6, 8 x 8192 x 4096 9.6
//                 / 12.6), but not few columns and a long K (1 x 512 x 8192 5.6 / 5.3)
//   to 16 rows    while K is short (16 x 512 x 2048 3.5 / 4.4, 16 x 8192 x 2048 7.1 /
//                 7.6), longer with many columns (16 x 2048 x 4096 5.6 / 5.8, 16 x 8192
//                 x 4096 11.1 / 12.0, but 16 x 512 x 4096 5.5 / 4.6 and 16 x 4096 x 8192
//                 10.2 / 9.5); from 16384 columns on about equal
//   to 32 rows    while B is small (32 x 2048 x 2048 3.5 / 4.7, 32 x 4096 x 1024 3.9 /
//                 4.7, 32 x 4096 x 2048 5.9 / 5.8), within two tiles of 16 columns for
//                 each SM (24 x 8192 x 512 5.1 / 4.3) and a short K (24 x 1024 x 4096
//                 5.1 / 4.8)
bool few_rows(long long M, long long N, long long K) {
  if (M <= 8) return N > 1024 || K < 8192;
  if (M <= 16) return K <= 2048 || (K <= 4096 && N >= 2048);
  return M <= kSkinnyRows && N <= 4864 && K <= 2048 && N * K <= (1LL << 22);
}

}  // namespace

cudaError_t launch_f8_gemm(const F8GemmArgs& a, DevPlan* plan, cudaStream_t st, int fault,
                           unsigned long long wait_ns) {
  const int variant = gemm_variant();
  if (variant == 0 && a.b_kmajor && few_rows(a.M, a.N, a.K))
    return launch_f8_skinny(a, plan, st);
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
  p.keep_status = a.keep_status;
  p.wait_ns = wait_ns;
  cudaLaunchAttribute attr[2];
  const long long tiles2 = ((a.M + 255) / 256) * ((a.N + BN2 - 1) / BN2);
  // Tiles of 128 x 128 while one wave of CTAs holds them all, split along K where
  // that leaves SMs idle; beyond that the pair kernel's tiles.  (4096 columns, K =
  // 4096: 512 rows, 128 tiles, 12.9 against the pairs' 19.3 us; 640 rows, 160
  // tiles, 24.8 against 19.9 us.)
  const bool pair = variant == 2 || (variant == 0 && (long long)p.mt * p.nt > fd.sms);
  const uint32_t b_cols = pair ? 64 : 128;  // columns of B per copy
  CUtensorMap ma, mb;
  if (!make_map_2d(&ma, dev, a.A, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.lda, BK, 128) ||
      !(a.b_kmajor ? make_map_2d(&mb, dev, a.B, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.ldb, BK, b_cols)
                   : make_map_2d(&mb, dev, a.B, (uint64_t)a.N, (uint64_t)a.K, (uint64_t)a.ldb, b_cols, BK,
                                 pair ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B)))
    return cudaErrorInvalidValue;
  if (pair) {
    p.mt = (int)((a.M + 255) / 256);
    p.nt = (int)((a.N + BN2 - 1) / BN2);
    const long long clusters = tiles2 < fd.max_pairs ? tiles2 : fd.max_pairs;
    cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)(2 * clusters)), NUM_THREADS, SMEM2_BYTES, st, 2, attr);
    CUtensorMap mc = {};
    if (p.vec_c && !make_map_2d(&mc, dev, a.C, (uint64_t)a.N, (uint64_t)a.M, (uint64_t)a.ldc * es, 64 / es, 32,
                                CU_TENSOR_MAP_SWIZZLE_64B,
                                es == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16))
      return cudaErrorInvalidValue;
    return cudaLaunchKernelEx(&cfg, kPairKernels[a.b_kmajor][a.tile_b], ma, mb, mc, p, plan);
  }
  const long long tiles = (long long)p.mt * p.nt;
  // Slices of K while all clusters are resident together (128 x 2048 x 4096: 13.5 us
  // in 16 clusters of eight, some of which wait for others to end, 7.4 in fours), of
  // at least four blocks: a slice of two saves less than its join costs (512 x 1024
  // x 1024 in four slices 6.0 us, in two 5.85; 1024 x 1024 x 512 in two 6.35, whole
  // 5.9).
  int S = 1;
  for (int i = 1; i < 4 && tiles <= fd.max_slices[i] && p.KB >= 8 * S; ++i) S *= 2;
  cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)(tiles * S)), NUM_THREADS, SMEM1_BYTES, st, S, attr);
  return cudaLaunchKernelEx(&cfg, kTileKernels[a.b_kmajor][a.tile_b], ma, mb, p, S, plan);
}

}  // namespace rg
