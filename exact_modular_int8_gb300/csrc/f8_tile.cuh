// f8_tile.cuh -- what the tensor-core products of block-scaled E4M3 matrices
// share: parameters, groups of rows, scales in shared memory, fp32 sums of the
// blocks' products and the host's tensor maps.  Included by one translation
// unit per kernel family.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "f8_act.cuh"
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

// Rows (or columns along the contraction) in groups; F8Groups as the kernels take it.
struct Groups {
  const void* offsets;  // [E + 1]
  int wide;             // 64-bit offsets
  int E;
  int limit;      // rows
  int zero_rest;  // write 0 to the rows behind the last group
};
constexpr int kMaxGroups = RG_MOE_MAX_EXPERTS;

struct Params {
  const float* SA;
  const float* SB;
  void* C;
  long long ldc, sa_ld, sb_n, sb_k, sb_e;
  int M, N, KB;
  int mt, nt;
  int out_type;
  int unit_c;  // rows of C (and P) start on boundaries of 16, 8, 4 or 2 bytes
  int fault;
  int keep_status;
  int late;
  unsigned long long wait_ns;
  F8Epilogue ep;
  int unit_r;  // the same of the residual
  Groups gr;
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
// any CTA could write to it.  Then the next kernel may start.  A late one that keeps
// the status has to find it cleared, and one thread that lets it start counts for its
// block: in the first block that is the clearing thread, once its stores are visible.
__device__ __forceinline__ void start_status(const Params& gp, DevPlan* plan) {
  if (blockIdx.x == 0 && !gp.keep_status) {
    if (threadIdx.x == 0) {
      plan->status = 0;
      plan->timeout_where = 0;
      __threadfence();
      allow_dependents();
    }
  } else {
    allow_dependents();
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
// [n0, n0 + NC), by NT threads t; SB: the scales of this B.  Entries past the
// matrix repeat its last.
template <int NC, bool TILE_B, int NT>
__device__ __forceinline__ void load_scales(const Params& gp, const float* SB, ScaleChunk<NC>& c, int m0, int n0,
                                            int kb0, int kb_end, int t) {
  const int kbi = t & (KC - 1), kb = min(kb0 + kbi, kb_end - 1);
#pragma unroll 4
  for (int r = t >> 3; r < 128; r += NT / 8)
    cp_async4(smem_u32(&c.a[kbi][r]), gp.SA + (long long)min(m0 + r, gp.M - 1) * gp.sa_ld + kb);
  if constexpr (TILE_B) {
    if (t < KC * (NC / 128)) {
      const int h = t >> 3;
      cp_async4(smem_u32(&c.b[kbi][h]),
                SB + (long long)min(n0 / 128 + h, (gp.N - 1) / 128) * gp.sb_n + kb * gp.sb_k);
    }
  } else if (gp.sb_k == 1) {
#pragma unroll 4
    for (int n = t >> 3; n < NC; n += NT / 8)
      cp_async4(smem_u32(&c.b[kbi][n]), SB + (long long)min(n0 + n, gp.N - 1) * gp.sb_n + kb);
  } else {
    for (int q = 0; q < KC; ++q)
      for (int n = t; n < NC; n += NT)
        cp_async4(smem_u32(&c.b[q][n]),
                  SB + (long long)min(n0 + n, gp.N - 1) * gp.sb_n + (long long)min(kb0 + q, kb_end - 1) * gp.sb_k);
  }
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
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
// Groups.  Each CTA reads the offsets into shared memory and numbers the tiles
// itself (E loads and one warp's scan), so that a product of groups is one
// launch whose offsets stay on the device.  rows[g] is where group g starts,
// first[g] its first tile; rows[E + 1] ends the rows behind the last group, which
// are a group without blocks when they are to be zero.
//
// Offsets that start above 0, fall, or end past the rows give no tile at all and
// RG_ERR_ARG as the call's status.  All threads call this, after the call's
// status has been cleared by the thread that reports.
// ---------------------------------------------------------------------------
struct GroupTable {
  int rows[kMaxGroups + 2];
  int first[kMaxGroups + 2];
};
__device__ __forceinline__ int offset_at(const Groups& gr, int i, bool& ok) {
  const long long v = gr.wide ? static_cast<const long long*>(gr.offsets)[i] : static_cast<const int*>(gr.offsets)[i];
  ok = ok && v >= 0 && v <= INT_MAX - 256;
  return (int)v;
}
// Along the contraction, group g's blocks of 128 start here.
__device__ __forceinline__ int first_block(int offset, int g) { return offset / 128 + g; }

// Tiles in all; tile_rows = 0: groups along the contraction, whose tiles need no numbering.
__device__ __forceinline__ int load_groups(const Groups& gr, GroupTable& tab, int tile_rows, int nt, DevPlan* plan) {
  bool ok = true;
  for (int i = threadIdx.x; i <= gr.E; i += blockDim.x) {
    const int v = offset_at(gr, i, ok);
    ok = ok && (i ? offset_at(gr, i - 1, ok) <= v : v == 0);
    if (i == gr.E) ok = ok && v <= gr.limit;
    tab.rows[i] = v;
  }
  if (threadIdx.x == 0) tab.rows[gr.E + 1] = gr.limit;
  ok = __syncthreads_and(ok);
  if (!ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(&plan->status, RG_ERR_ARG);
    return 0;
  }
  if (!tile_rows) return 1;
  const int n = gr.E + (gr.zero_rest ? 1 : 0);
  if (threadIdx.x < 32) {  // a lane numbers `per` groups in a row
    const int lane = threadIdx.x, per = (n + 31) / 32, g0 = min(lane * per, n), g1 = min(g0 + per, n);
    int sum = 0;
    for (int g = g0; g < g1; ++g) sum += (tab.rows[g + 1] - tab.rows[g] + tile_rows - 1) / tile_rows * nt;
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
      if (lane >= o) before += v;
    }
    before -= sum;
    for (int g = g0; g < g1; ++g) {
      tab.first[g] = before;
      before += (tab.rows[g + 1] - tab.rows[g] + tile_rows - 1) / tile_rows * nt;
    }
    if (g1 == n && g0 < n) tab.first[n] = before;
  }
  __syncthreads();
  return tab.first[n];
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

// The same of matrices one behind the other, `stride2` bytes apart; a copy is cut to its own matrix.
bool make_map_stack(CUtensorMap* m, int dev, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                    uint64_t stride_bytes, uint64_t stride2, uint32_t b0, uint32_t b1,
                    CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {stride_bytes, stride2};
  cuuint32_t box[3] = {b0, b1, 1};
  cuuint32_t es[3] = {1, 1, 1};
  auto encode = [&] {
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

}  // namespace
}  // namespace rg
