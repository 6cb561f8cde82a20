// f8_grouped.cu -- products of block-scaled E4M3 matrices by group: rows sorted
// by expert with a weight matrix for each (outputs and input gradients), and
// sums over each expert's rows (weight gradients).
//
// With many rows to an expert the CTA-pair kernel walks the groups' tiles of 256
// x 256 (f8_pair.cuh).  With few, the work is reading the experts' weights once,
// and a tile of 256 rows would be padding: the kernel below turns the product
// round.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include "f8_pair.cuh"

namespace rg {
namespace {

// ---------------------------------------------------------------------------
// Few rows to a group.  The weights' columns n are the 128 rows of the MMA and
// the group's rows (tokens) its columns, 16 to 128 of them as there are: D[n][t],
// so that neither the MMA nor the read-back nor the copies are padded to more than
// 16 tokens (32 for the copies).  An epilogue warp holds 32 n x every other 16
// tokens; its lanes store neighbouring n, whole sectors of C.
//
// Persistent, a CTA per SM: a unit is 128 columns of one group's weights times up
// to 128 of its tokens, over all of K.  The producer runs up to six blocks (of 16
// KB of weights) ahead, across units, which is what keeps the weights coming.
//
// Sixteen epilogue warps with an instance of their loop for each number of 16-token
// parts, and scales that reach them multiplied.  8 groups of 2048 x 4096, operands in
// L2, 1 and 128 tokens to a group: 14.3 and 20.9 us, of which each block of k takes
// 0.31 and 0.44; with an empty epilogue 11.7 and 17.4, which is L2's rate of 11 TB/s.
// Eight warps took 13.7 and 23.1, with parts skipped at run time and the scales
// multiplied in the loop 15.5 and 26.5 (parts that are not there still cost their
// moves), two blocks to a barrier 16.1 and 30.5.  64 groups of 2048 x 2048 from memory,
// 1 token each: 45.4 us, 5.9 TB/s.
// ---------------------------------------------------------------------------
constexpr int NTOK = 128;
constexpr int TOK_BOX = 32;  // tokens per copy
constexpr int STAGES_N = 6;
constexpr int STAGE_N_BYTES = 2 * SLAB;
constexpr int ACCS = 4;  // accumulators: all of tensor memory
constexpr int SETS = 4;  // of four epilogue warps: every SETS-th 16 tokens each
constexpr int SUM_WARPS = 4 * SETS;
constexpr int FEW_THREADS = 128 + 32 * SUM_WARPS;
struct TokenScales {
  float s[KC][NTOK + 4];  // token's times the weights'
};
constexpr int SCALE_N_BYTES = SCALE_BUFS * (int)sizeof(TokenScales);
constexpr int SMEM_N_BYTES = 1024 + STAGES_N * STAGE_N_BYTES + SCALE_N_BYTES + 256 + (int)sizeof(GroupTable);
static_assert(SMEM_N_BYTES <= 232448, "shared memory");

// Unit t: rows [m0, m0 + count) of A and C, columns from n0 on, group g.
struct UnitAt {
  int m0, count, n0, kb1, g;
};
struct Units {
  const Params& gp;
  const GroupTable& tab;
  int g = 0;
  // t grows from call to call
  __device__ __forceinline__ UnitAt at(int t) {
    while (t >= tab.first[g + 1]) ++g;
    const int row = tab.rows[g], rows = tab.rows[g + 1] - row, parts = (rows + NTOK - 1) / NTOK, i = t - tab.first[g];
    const int tn = i / parts, part = i - tn * parts;
    // parts of equal size: at most 128, so that the last holds at least one
    const int each = ((rows + parts - 1) / parts + 15) & ~15;
    return UnitAt{row + part * each, min(each, rows - part * each), tn * 128, g < gp.gr.E ? gp.KB : 0, g};
  }
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : RG_R8(0), RG_R8(8)
      : "r"(taddr));
}

// An epilogue warp's place in the pipeline.
struct UnitPipe {
  uint64_t *done, *tempty, *sfull, *sempty;
  const TokenScales* scales;
  uint32_t it, phase;
  int chunk, st;  // chunks of scales, pipeline stage
  bool ok;        // the same for all lanes
};

// One unit's sums of 32 columns from n0 on and PARTS times 16 tokens, every
// SETS-th 16 from 16 `set` on, and their way to C.
template <int PARTS>
__device__ __forceinline__ void sum_unit(const Params& gp, const UnitAt& at, UnitPipe& p, uint32_t lane_addr, int set,
                                         int n0, int lane, const Ctl& ctl) {
  constexpr int P = PARTS ? PARTS : 1;
  uint64_t acc[P][8] = {};
  for (int kb = 0; kb < at.kb1; ++kb) {
    const uint32_t b = p.it % ACCS;
    const int kbi = kb % KC;
    bool ok = kbi != 0 || wait_bounded(smem_u32(&p.sfull[p.chunk & 1]), (p.chunk >> 1) & 1u, ctl, 46);
    p.ok = __all_sync(0xFFFFFFFFu, ok && wait_bounded(smem_u32(&p.done[p.st]), p.phase, ctl, 44));
    if (++p.st == STAGES_N) {
      p.st = 0;
      p.phase ^= 1u;
    }
    ++p.it;
    if (!p.ok) return;
    tc_fence_after();
    uint32_t r[P][16];
#pragma unroll
    for (int i = 0; i < PARTS; ++i) tmem_ld16(lane_addr + b * NTOK + 16 * SETS * i, r[i]);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(r[i][j]));
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_relaxed(smem_u32(&p.tempty[b]));
    const float* s = p.scales[p.chunk & 1].s[kbi] + set * 16;
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(s + 16 * SETS * i + 2 * j);
        acc[i][j] = fma2(pack2u(r[i][2 * j], r[i][2 * j + 1]), w.x, acc[i][j]);
        acc[i][j + 1] = fma2(pack2u(r[i][2 * j + 2], r[i][2 * j + 3]), w.y, acc[i][j + 1]);
      }
    if (kbi == KC - 1 || kb == at.kb1 - 1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p.sempty[p.chunk & 1]));
      ++p.chunk;
    }
  }
  const int n = n0 + lane;
  if (n < gp.N) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int first = 16 * SETS * i + set * 16, left = at.count - first;
      const long long out = (long long)(at.m0 + first) * gp.ldc + n;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = unpack2(acc[i][j]);
        if (2 * j < left) store_real(gp.C, gp.out_type, out + 2 * j * gp.ldc, f.x);
        if (2 * j + 1 < left) store_real(gp.C, gp.out_type, out + (2 * j + 1) * gp.ldc, f.y);
      }
    }
  }
}

template <bool B_KMAJOR>
__global__ void __launch_bounds__(FEW_THREADS, 1)
    f8_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ Params gp, DevPlan* plan) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stage_base = smem;  // weights, then tokens
  TokenScales* scales = reinterpret_cast<TokenScales*>(smem + STAGES_N * STAGE_N_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES_N * STAGE_N_BYTES + SCALE_N_BYTES);
  uint64_t* full = bars;
  uint64_t* done = bars + STAGES_N;        // the stage's MMAs are complete
  uint64_t* tempty = bars + 2 * STAGES_N;  // by accumulator
  uint64_t* sfull = tempty + ACCS;
  uint64_t* sempty = sfull + SCALE_BUFS;
  uint64_t* drain = sempty + SCALE_BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  GroupTable& tab = *reinterpret_cast<GroupTable*>(reinterpret_cast<uint8_t*>(bars) + 256);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ctl ctl{abort_flag, &plan->status, &plan->timeout_where, gp.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES_N; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&done[s]), 1);
    }
    for (int b = 0; b < ACCS; ++b) mbar_init(smem_u32(&tempty[b]), SUM_WARPS);
    for (int b = 0; b < SCALE_BUFS; ++b) {
      mbar_init(smem_u32(&sfull[b]), 64);
      mbar_init(smem_u32(&sempty[b]), SUM_WARPS);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"((uint32_t)(ACCS * NTOK)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // the set-up above overlaps the predecessor's tail
  if (!gp.late) wait_for_predecessor();
  start_status(gp, plan);
  const int total = load_groups(gp.gr, tab, NTOK, gp.nt, plan);
  Units units{gp, tab};

  if (warp < 4) {
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      bool issued[STAGES_N] = {};
      uint32_t issued_phase[STAGES_N] = {};
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const UnitAt at = units.at(t);
        const int boxes = (at.count + TOK_BOX - 1) / TOK_BOX;
        for (int kb = 0; kb < at.kb1; ++kb) {
          if (!wait_bounded(smem_u32(&done[stage]), phase ^ 1u, ctl, 41)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full[stage]);
          mbar_arrive_expect_tx(fb, (uint32_t)(SLAB + boxes * TOK_BOX * BK));
          const uint32_t b_dst = smem_u32(stage_base + stage * STAGE_N_BYTES);
          if constexpr (B_KMAJOR) tma_load_3d(b_dst, &tmB, fb, kb * BK, at.n0, at.g);
          else tma_load_3d(b_dst, &tmB, fb, at.n0, kb * BK, at.g);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(b_dst + SLAB + i * TOK_BOX * BK, &tmA, fb, kb * BK, at.m0 + i * TOK_BOX);
          issued[stage] = true;
          issued_phase[stage] = phase;
          if (++stage == STAGES_N) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {  // let issued copies land before the block exits
        Ctl drain_ctl = ctl;
        volatile int never = 0;
        drain_ctl.abort = &never;
        for (int s = 0; s < STAGES_N; ++s)
          if (issued[s]) wait_bounded(smem_u32(&full[s]), issued_phase[s], drain_ctl, 0);
      }
    }
    if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t w_addr = smem_u32(stage_base), x_addr = w_addr + SLAB;
      const uint64_t wdesc0 = B_KMAJOR ? sw128_desc(w_addr, 16, 1024) : sw128_desc(w_addr, SLAB, 1024);
      const uint64_t xdesc0 = sw128_desc(x_addr, 16, 1024);
      constexpr uint32_t w_step = B_KMAJOR ? 2 : 256;  // 32 k: 32 bytes along a row, or 32 rows of 128 bytes
      int stage = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const UnitAt at = units.at(t);
        // the weights are the A operand: M-major where they lie [K][N]
        const uint32_t idesc = idesc_f8(128, (at.count + 15) & ~15, true) | (B_KMAJOR ? 0u : 1u << 15);
        for (int kb = 0; kb < at.kb1; ++kb, ++it) {
          const uint32_t b = it % ACCS, aph = (it / ACCS) & 1u;
          ok = wait_both(smem_u32(&tempty[b]), aph ^ 1u, smem_u32(&full[stage]), phase, ctl, 42);
          if (!ok) break;
          tc_fence_after();
          const uint64_t off = (uint64_t)(stage * (STAGE_N_BYTES >> 4));
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)
              umma_f8(tmem_base + b * NTOK, wdesc0 + off + (uint64_t)(w_step * kk), xdesc0 + off + (uint64_t)(2 * kk),
                      idesc, kk > 0);
            if (!(gp.fault == 1 && it == 0)) umma_commit(smem_u32(&done[stage]));
          }
          __syncwarp();
          if (++stage == STAGES_N) {
            stage = 0;
            phase ^= 1u;
          }
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
    }
    if (warp >= 2) {
      // ---------------------------------------------------------- scales
      const int tid = threadIdx.x - 64, kbi = tid & (KC - 1);
      int c = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const UnitAt at = units.at(t);
        const float* SB = gp.SB + at.g * gp.sb_e + at.n0 / 128 * gp.sb_n;
        for (int kb0 = 0; kb0 < at.kb1; kb0 += KC, ++c) {
          const int b = c & 1, kb = min(kb0 + kbi, at.kb1 - 1);
          ok = wait_bounded(smem_u32(&sempty[b]), ((c >> 1) & 1u) ^ 1u, ctl, 45);
          if (!ok) break;
          const float sb = SB[kb * gp.sb_k];
          const float* sa = gp.SA + (long long)at.m0 * gp.sa_ld + kb;
          float v[NTOK / 8];  // all under way before the first is stored
#pragma unroll
          for (int i = 0; i < NTOK / 8; ++i) {
            const int r = (tid >> 3) + 8 * i;
            v[i] = r < at.count ? __ldg(sa + r * gp.sa_ld) : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < NTOK / 8; ++i)
            if ((tid >> 3) + 8 * i < at.count) scales[b].s[kbi][(tid >> 3) + 8 * i] = v[i] * sb;
          mbar_arrive(smem_u32(&sfull[b]));
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q4 = warp & 3;           // tensor-memory lane quarter this warp may access
    const int set = (warp - 4) >> 2;
    static_assert(NTOK == 2 * 16 * SETS, "up to two parts to a warp");
    const uint32_t lane_addr = tmem_base + ((uint32_t)(q4 * 32) << 16) + set * 16;
    UnitPipe pipe{full + STAGES_N, tempty, sfull, sempty, scales, 0, 0, 0, 0, true};
    for (int t = blockIdx.x; t < total && pipe.ok; t += gridDim.x) {
      const UnitAt at = units.at(t);
      const int n0 = at.n0 + q4 * 32;
      // 16-token parts with a token: an instance for each number, whose loops are unrolled
      switch ((at.count - set * 16 + 16 * SETS - 1) / (16 * SETS)) {
        case 0: sum_unit<0>(gp, at, pipe, lane_addr, set, n0, lane, ctl); break;
        case 1: sum_unit<1>(gp, at, pipe, lane_addr, set, n0, lane, ctl); break;
        default: sum_unit<2>(gp, at, pipe, lane_addr, set, n0, lane, ctl); break;
      }
    }
  }

  __syncwarp();
  if (gp.late) wait_for_predecessor();
  if (*abort_flag) {  // products that no role has waited for: give them time to end
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"((uint32_t)(ACCS * NTOK)));
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using FewKernel = void (*)(const CUtensorMap, const CUtensorMap, const Params, DevPlan*);
constexpr FewKernel kFewKernels[2] = {f8_few_kernel<false>, f8_few_kernel<true>};
constexpr PairKernel kRowsKernels[2] = {f8_gemm_pair_kernel<false, true, WALK_ROWS, PLAIN, false, false>,
                                        f8_gemm_pair_kernel<true, true, WALK_ROWS, PLAIN, false, false>};
constexpr PairKernel kBlocksKernel = f8_gemm_pair_kernel<true, false, WALK_BLOCKS, PLAIN, false, false>;

struct GroupedDevice {
  int sms = 0, max_pairs = 0;
};
cudaError_t grouped_device(int dev, GroupedDevice& out) {
  static std::mutex mu;
  static GroupedDevice devs[64];
  std::lock_guard<std::mutex> lock(mu);
  GroupedDevice& d = devs[dev];
  if (!d.sms) {
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
      e = cudaFuncSetAttribute(kFewKernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_N_BYTES);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kRowsKernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 pair_smem(WALK_ROWS, PLAIN));
    }
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kBlocksKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pair_smem(WALK_BLOCKS, PLAIN));
    if (e != cudaSuccess) return e;
    if (sms < 2) return cudaErrorInvalidDevice;
    // not every SM can be paired within its GPC
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)(sms & ~1)), NUM_THREADS, pair_smem(WALK_ROWS, PLAIN), nullptr,
                                            2, attr);
    if (cudaOccupancyMaxActiveClusters(&d.max_pairs, reinterpret_cast<const void*>(kRowsKernels[1]), &cfg) !=
            cudaSuccess ||
        d.max_pairs < 1) {
      cudaGetLastError();  // the query's own failure is not the call's
      d.max_pairs = sms / 2;
    }
    d.sms = sms;
  }
  out = d;
  return cudaSuccess;
}

// Which kernel, by the time that each would take: waves of its tiles, of which half
// a one is lost to each group (but a group has at least one), times what a tile
// takes.  The few-row kernel's blocks take 0.28 us with a token and 0.44 with 128, the
// pairs' 0.53, and a tile 0.8 and 2.5 more.  (Alone a block with a token takes 0.31, as
// above; either value chooses alike in every row below.)  T is all rows of A, those
// behind the last group among them, since the offsets are on the device: a few rows in
// a buffer with room for many go to the pairs.  Measured, us, few-row kernel first (groups
// of uneven sizes; E x N x K, rows to a group on average):
//   64 x 2048 x 4096  8: 88 / 137   64: 115 / 139   96: 142 / 154   128: 158 / 156
//                     256: 276 / 212   1024: 922 / 575
//   16 x 1544 x 2056  312: 49 / 38;   16 x 1024 x 1024  250: 14.6 / 16.3
//   8 x 1024 x 1024   128: 9.2 / 9.8
bool few_rows_to_a_group(long long T, long long E, long long N, long long KB, int sms, int pairs) {
  const long long G = std::min(E, T);
  auto tiles = [&](long long rows, long long cols) {
    return std::max(G, T / rows + G / 2) * ((N + cols - 1) / cols);
  };
  const double waves_few = (double)((tiles(NTOK, 128) + sms - 1) / sms);
  const double waves_pair = (double)((tiles(256, BN2) + pairs - 1) / pairs);
  const double tokens = std::min(1.0, (double)T / (double)(G * NTOK));
  return waves_few * ((0.28 + 0.16 * tokens) * (double)KB + 0.8) < waves_pair * (0.53 * (double)KB + 2.5);
}

}  // namespace

cudaError_t launch_f8_grouped(const F8GemmArgs& a, const F8Groups& g, DevPlan* plan, cudaStream_t st, int fault,
                              unsigned long long wait_ns) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  GroupedDevice gd;
  e = grouped_device(dev, gd);
  if (e != cudaSuccess) return e;
  const int es = a.out_type == RG_TYPE_F32 ? 4 : 2, variant = gemm_variant();
  Params p = {};
  p.SA = a.SA;
  p.SB = a.SB;
  p.C = a.C;
  p.ldc = a.ldc;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.KB = (int)((a.K + BK - 1) / BK);
  p.sa_ld = p.KB;
  p.sb_n = a.sb_n;
  p.sb_k = a.sb_k;
  p.sb_e = (long long)p.KB * ((a.N + 127) / 128);
  p.out_type = a.out_type;
  p.unit_c = row_unit(a.C, a.ldc * es);
  p.fault = fault;
  p.keep_status = a.keep_status;
  p.late = a.late;
  p.wait_ns = wait_ns;
  p.gr = Groups{g.offsets, g.wide, (int)g.E, (int)g.rows, g.zero_rest};
  const bool few = !g.by_blocks && (variant == 1 || (variant == 0 && few_rows_to_a_group(a.M, g.E, a.N, p.KB, gd.sms,
                                                                                         gd.max_pairs)));
  // groups that can have a row, and the rows behind them
  const long long groups = std::min(g.E, a.M) + 1;
  cudaLaunchAttribute attr[2];
  CUtensorMap ma, mb, mc = {}, mp = {};
  if (!g.by_blocks) {
    const uint32_t cols = few ? 128 : 64;  // columns of B per copy
    if (!(a.b_kmajor ? make_map_stack(&mb, dev, a.B, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)g.E, (uint64_t)a.ldb,
                                      (uint64_t)(a.ldb * a.N), BK, cols)
                     : make_map_stack(&mb, dev, a.B, (uint64_t)a.N, (uint64_t)a.K, (uint64_t)g.E, (uint64_t)a.ldb,
                                      (uint64_t)(a.ldb * a.K), cols, BK,
                                      few ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B)))
      return cudaErrorInvalidValue;
  }
  if (few) {
    p.nt = (int)((a.N + 127) / 128);
    if (!make_map_2d(&ma, dev, a.A, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.lda, BK, TOK_BOX))
      return cudaErrorInvalidValue;
    const long long units = (a.M / NTOK + groups) * p.nt;
    return launch_dependent(kFewKernels[a.b_kmajor], dim3((unsigned)std::min<long long>(units, gd.sms)),
                            dim3(FEW_THREADS), SMEM_N_BYTES, st, ma, mb, p, plan);
  }
  p.nt = (int)((a.N + BN2 - 1) / BN2);
  long long tiles = (a.M / 256 + groups) * p.nt;
  PairKernel kernel = kRowsKernels[a.b_kmajor];
  if (g.by_blocks) {
    p.mt = (int)((a.M + 255) / 256);
    tiles = g.E * p.mt * p.nt;
    kernel = kBlocksKernel;
    if (!make_map_2d(&mb, dev, a.B, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.ldb, BK, 64)) return cudaErrorInvalidValue;
  }
  if (!pair_maps(a, p, dev, &ma, &mc, &mp, g.by_blocks ? g.E * a.M : a.M)) return cudaErrorInvalidValue;
  const long long clusters = std::min<long long>(tiles, gd.max_pairs);
  cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)(2 * clusters)), NUM_THREADS,
                                          pair_smem(g.by_blocks ? WALK_BLOCKS : WALK_ROWS, PLAIN), st, 2, attr);
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, mc, mp, p, plan);
}

}  // namespace rg
