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
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include "f8_pair.cuh"

namespace rg {
namespace {

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

// Four neighbouring entries of a row, `left` of them in the matrix; vec: they lie on a boundary of their size.
__device__ __forceinline__ void put4(void* p, long long at, int type, int vec, int left, const float (&e)[4]) {
  if (vec && left >= 4) {
    if (type == RG_TYPE_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(e[0], e[1], e[2], e[3]);
    } else {
      uint2 w;
      if (type == RG_TYPE_F16) {
        const __half2 a = __floats2half2_rn(e[0], e[1]), b = __floats2half2_rn(e[2], e[3]);
        w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(e[0], e[1]), b = __floats2bfloat162_rn(e[2], e[3]);
        w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) = w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < left) store_real(p, type, at + q, e[q]);
  }
}
__device__ __forceinline__ int four_at_once(int unit, int type) { return unit >= (type == RG_TYPE_F32 ? 16 : 8); }

// What the epilogue needs of the parameters, by value.
struct Finish {
  void *C, *P;
  int out_type, act, vec;
  float4 bias;
};
__device__ __forceinline__ float entry(const uint4& w, int type, int q) {  // of four, as loaded
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  if (type == RG_TYPE_F32) return __uint_as_float(v[q]);
  const uint32_t h = v[q >> 1] >> (16 * (q & 1));
  return type == RG_TYPE_F16 ? __half2float(__ushort_as_half((unsigned short)h)) : __uint_as_float(h << 16);
}
// Four entries of a row, `left` of them in the matrix, through the epilogue; res: the
// residual's.  Not inlined: a warp's rows share its code, whose fetching is what a
// small product would wait for (512 x 1024 x 1024 with a bias: 7.7 us, inlined 12.2; 5.9
// without an epilogue).
__device__ __noinline__ void finish4(Finish f, long long out, int left, float4 v, uint4 res) {
  float e[4] = {v.x + f.bias.x, v.y + f.bias.y, v.z + f.bias.z, v.w + f.bias.w};
  if (f.P) put4(f.P, out, f.out_type, f.vec, left, e);
  switch (f.act) {
    case RG_ACT_RELU:
      for (float& x : e) x = activate<RG_ACT_RELU>(x);
      break;
    case RG_ACT_SILU:
      for (float& x : e) x = activate<RG_ACT_SILU>(x);
      break;
    case RG_ACT_GELU:
      for (float& x : e) x = activate<RG_ACT_GELU>(x);
      break;
    case RG_ACT_GELU_TANH:
      for (float& x : e) x = activate<RG_ACT_GELU_TANH>(x);
      break;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) e[q] += entry(res, f.out_type, q);
  put4(f.C, out, f.out_type, f.vec, left, e);
}
__device__ __forceinline__ Finish make_finish(const Params& gp, int n, int left) {
  Finish f = {gp.C, gp.ep.P, gp.out_type, gp.ep.act, four_at_once(gp.unit_c, gp.out_type), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  if (gp.ep.bias) {
    if (left > 0) f.bias.x = load_real(gp.ep.bias, gp.ep.bias_type, n);
    if (left > 1) f.bias.y = load_real(gp.ep.bias, gp.ep.bias_type, n + 1);
    if (left > 2) f.bias.z = load_real(gp.ep.bias, gp.ep.bias_type, n + 2);
    if (left > 3) f.bias.w = load_real(gp.ep.bias, gp.ep.bias_type, n + 3);
  }
  return f;
}
// The residual's four entries from `at` on, as entry() takes them; zeros without one.
__device__ __forceinline__ uint4 load_residual4(const Params& gp, long long at, int left) {
  uint4 w = make_uint4(0, 0, 0, 0);
  if (!gp.ep.R) return w;
  if (four_at_once(gp.unit_r, gp.out_type) && left >= 4) {
    if (gp.out_type == RG_TYPE_F32) return *reinterpret_cast<const uint4*>(static_cast<const float*>(gp.ep.R) + at);
    const uint2 h = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(gp.ep.R) + at);
    return make_uint4(h.x, h.y, 0, 0);
  }
  uint32_t v[4] = {};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q < left) {
      if (gp.out_type == RG_TYPE_F32) v[q] = static_cast<const uint32_t*>(gp.ep.R)[at + q];
      else v[q >> 1] |= (uint32_t)static_cast<const uint16_t*>(gp.ep.R)[at + q] << (16 * (q & 1));
    }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Rows rank, rank + S, ... of the tile: the slices' sums in rank order.  A warp
// fetches all of its rows (S = 1: half of them) from every slice before it adds
// the first, so that the way to another CTA's shared memory, most of a
// microsecond, is waited for once.  The CTAs part when their reads are done,
// before their stores to C.
template <int S, bool EPI>
__device__ __forceinline__ void join_slices(const Params& gp, uint32_t part, int rank, int tm, int tn, int warp, int lane,
                                            bool live, const Finish& f) {
  constexpr int WARPS = NUM_THREADS / 32, ROWS = (128 / S + WARPS - 1) / WARPS, R = S == 1 ? (ROWS + 1) / 2 : ROWS;
  const int rows = min(128, gp.M - tm * 128), cols = min(BN1, gp.N - tn * BN1);
  const int c = 4 * lane;  // this lane's columns
#pragma unroll
  for (int i0 = 0; i0 < ROWS; i0 += R) {
    float4 v[S][R];
    uint4 res[EPI ? R : 1];
    if constexpr (EPI) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = rank + S * (warp + WARPS * (i0 + i));
        res[i] = make_uint4(0, 0, 0, 0);
        if (live && r < rows && c < cols)
          res[i] = load_residual4(gp, (long long)(tm * 128 + r) * gp.ep.ldr + tn * BN1 + c, cols - c);
      }
    }
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
      if (live && r < rows && c < cols) {
        const long long out = (long long)(tm * 128 + r) * gp.ldc + (long long)tn * BN1 + c;
        if constexpr (EPI) finish4(f, out, cols - c, v[0][i], res[i]);
        else put4(gp.C, out, gp.out_type, four_at_once(gp.unit_c, gp.out_type), cols - c,
                   {v[0][i].x, v[0][i].y, v[0][i].z, v[0][i].w});
      }
    }
  }
  __syncwarp();
  if (S > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <bool B_KMAJOR, bool TILE_B, bool EPI>
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
  if (!gp.late) wait_for_predecessor();
  start_status(gp, plan);

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
      load_scales<BN1, TILE_B, 64>(gp, gp.SB, scales[b], tm * 128, tn * BN1, kb, kb_hi, threadIdx.x - 64);
      cp_async_arrive(smem_u32(&sfull[b]));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------------------------------------ epilogue
    if constexpr (EPI) {  // the tile's residual to L2
      const int row = tm * 128 + (threadIdx.x >> 1) - 64, n0 = tn * BN1, es = gp.out_type == RG_TYPE_F32 ? 4 : 2;
      const int bytes = min(BN1, gp.N - n0) * es;
      if (gp.ep.R && row < gp.M)
        for (int i = 128 * (threadIdx.x & 1); i < bytes; i += 256)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(gp.ep.R) +
                                                         ((long long)row * gp.ep.ldr + n0) * es + i));
    }
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
  Finish f = {};
  if constexpr (EPI) f = make_finish(gp, tn * BN1 + 4 * lane, gp.N - tn * BN1 - 4 * lane);  // under way as the CTAs meet
  if (gp.late) wait_for_predecessor();
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
  if (S == 1) join_slices<1, EPI>(gp, part, rank, tm, tn, warp, lane, live, f);
  else if (S == 2) join_slices<2, EPI>(gp, part, rank, tm, tn, warp, lane, live, f);
  else if (S == 4) join_slices<4, EPI>(gp, part, rank, tm, tn, warp, lane, live, f);
  else join_slices<8, EPI>(gp, part, rank, tm, tn, warp, lane, live, f);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using TileKernel = void (*)(const CUtensorMap, const CUtensorMap, const Params, int, DevPlan*);
constexpr TileKernel kTileKernels[2][2] = {
    {f8_gemm_tile_kernel<false, false, false>, f8_gemm_tile_kernel<false, true, false>},
    {f8_gemm_tile_kernel<true, false, false>, f8_gemm_tile_kernel<true, true, false>}};
constexpr TileKernel kTileActKernel = f8_gemm_tile_kernel<true, true, true>;

template <bool B_KMAJOR, bool TILE_B>
constexpr PairKernel kWhole = f8_gemm_pair_kernel<B_KMAJOR, TILE_B, WALK_WHOLE, PLAIN, false, false>;
constexpr PairKernel kPairKernels[2][2] = {{kWhole<false, false>, kWhole<false, true>},
                                           {kWhole<true, false>, kWhole<true, true>}};
constexpr int SMEM2_BYTES = pair_smem(WALK_WHOLE, PLAIN);

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
    cudaError_t set = cudaFuncSetAttribute(kTileActKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM1_BYTES);
    for (int i = 0; i < 4 * (RG_ACT_GELU_TANH + 1) && set == cudaSuccess; ++i)
      set = cudaFuncSetAttribute((i & 2 ? pair_act_ragged_kernel : pair_act_kernel)(i >> 2, i & 1),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, pair_smem(WALK_WHOLE, SIMPLE_ACT));
    if (set != cudaSuccess) return set;
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
  Params p = {};
  p.SA = a.SA;
  p.SB = a.SB;
  p.C = a.C;
  p.ldc = a.ldc;
  p.sb_n = a.sb_n;
  p.sb_k = a.sb_k;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.KB = (int)((a.K + BK - 1) / BK);
  p.sa_ld = p.KB;
  p.mt = (int)((a.M + 127) / 128);
  p.nt = (int)((a.N + BN1 - 1) / BN1);
  p.out_type = a.out_type;
  const int es = a.out_type == RG_TYPE_F32 ? 4 : 2;
  p.unit_c = row_unit(a.C, a.ldc * es);
  p.fault = fault;
  p.keep_status = a.keep_status;
  p.late = a.late;
  p.wait_ns = wait_ns;
  if (a.ep) {
    p.ep = *a.ep;
    p.unit_c = std::min(p.unit_c, row_unit(a.ep->P, a.ldc * es));
    p.unit_r = row_unit(a.ep->R, a.ep->ldr * es);
  }
  cudaLaunchAttribute attr[2];
  const long long tiles2 = ((a.M + 255) / 256) * ((a.N + BN2 - 1) / BN2);
  // Tiles of 128 x 128 while one wave of CTAs holds them all, split along K where
  // that leaves SMs idle; beyond that the pair kernel's tiles.  (4096 columns, K =
  // 4096: 512 rows, 128 tiles, 12.9 against the pairs' 19.3 us; 640 rows, 160
  // tiles, 24.8 against 19.9 us.)
  const bool pair = variant == 2 || (variant == 0 && (long long)p.mt * p.nt > fd.sms);
  const uint32_t b_cols = pair ? 64 : 128;  // columns of B per copy
  CUtensorMap ma, mb;
  if (!(a.b_kmajor ? make_map_2d(&mb, dev, a.B, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.ldb, BK, b_cols)
                   : make_map_2d(&mb, dev, a.B, (uint64_t)a.N, (uint64_t)a.K, (uint64_t)a.ldb, b_cols, BK,
                                 pair ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B)))
    return cudaErrorInvalidValue;
  if (pair) {
    p.mt = (int)((a.M + 255) / 256);
    p.nt = (int)((a.N + BN2 - 1) / BN2);
    const long long clusters = tiles2 < fd.max_pairs ? tiles2 : fd.max_pairs;
    cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)(2 * clusters)), NUM_THREADS,
                                            pair_smem(WALK_WHOLE, a.ep ? SIMPLE_ACT : PLAIN), st, 2, attr);
    CUtensorMap mc = {}, mp = {};
    if (!pair_maps(a, p, dev, &ma, &mc, &mp, a.M)) return cudaErrorInvalidValue;
    PairKernel kernel = kPairKernels[a.b_kmajor][a.tile_b];
    if (a.ep) {
      const bool ragged = p.unit_c < 16 || (p.ep.R && (p.unit_r < 16 || a.N * es % 16 != 0));
      const void* act = (ragged ? pair_act_ragged_kernel : pair_act_kernel)(a.ep->act, a.ep->R);
      kernel = reinterpret_cast<PairKernel>(const_cast<void*>(act));
    }
    return cudaLaunchKernelEx(&cfg, kernel, ma, mb, mc, mp, p, plan);
  }
  if (!make_map_2d(&ma, dev, a.A, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.lda, BK, 128)) return cudaErrorInvalidValue;
  const long long tiles = (long long)p.mt * p.nt;
  // Slices of K while all clusters are resident together (128 x 2048 x 4096: 13.5 us
  // in 16 clusters of eight, some of which wait for others to end, 7.4 in fours), of
  // at least four blocks: a slice of two saves less than its join costs (512 x 1024
  // x 1024 in four slices 6.0 us, in two 5.85; 1024 x 1024 x 512 in two 6.35, whole
  // 5.9).
  int S = 1;
  for (int i = 1; i < 4 && tiles <= fd.max_slices[i] && p.KB >= 8 * S; ++i) S *= 2;
  cudaLaunchConfig_t cfg = cluster_config(dim3((unsigned)(tiles * S)), NUM_THREADS, SMEM1_BYTES, st, S, attr);
  return cudaLaunchKernelEx(&cfg, a.ep ? kTileActKernel : kTileKernels[a.b_kmajor][a.tile_b], ma, mb, p, S, plan);
}

}  // namespace rg