// f8_pair.cuh -- the persistent CTA-pair kernel of block-scaled E4M3 products:
// whole matrices, matrices by groups of rows, and groups along the contraction;
// with or without an epilogue.
#pragma once
#include "f8_tile.cuh"

namespace rg {
namespace {

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
// cycles a block (380 us with fp32 results); 2048 x 4096 x 8100 108 us.  (16 warps whose
// registers hold, 56 and 104 of them, 64 columns each: 271 us; with a scale for each
// of B's rows, where tensor memory gives fragments 250 bytes a cycle, 360 us.)
//
// With an epilogue, 8192 x 8192 x 2048 bf16 (133 us without): a bias 141 us, silu 159,
// gelu 172, residual 164, values before the activation 154, gelu with all of these 211.
// The epilogue warps do it while no sums are made, so its instructions and waits
// count whole: biases come through the scales' warp (fetched by the epilogue warps:
// 152 us), activations are 5 to 13 operations (gelu by erff: 214), the residual comes
// through a ring (loads by the lanes spilled in the blocks' loop: 323).
//
// The block is launched with 168 registers a thread; the first warpgroup
// (producer, MMA issue, scales) gives up 112 of them and the two epilogue
// warpgroups take 56 more each: 56 + 2 * 224 = 3 * 168.
// ---------------------------------------------------------------------------
constexpr int BN2 = 256;
constexpr int STAGES2 = 5;
constexpr int STAGES2_RING = 4;  // with a residual, whose rings take a stage's place
constexpr int STAGE2_BYTES = 2 * SLAB;
constexpr int HALF_SLAB = SLAB / 2;  // a CTA's 64 columns of one half
constexpr int PAIR_COLS = BN2 * 4 / EPI_WARPS;  // columns per epilogue warp
constexpr int OUT_BUF = 32 * 64;  // 64 bytes of each of a warp's rows
constexpr int OUT_WARP = 2 * OUT_BUF;
constexpr int SCALE2_BYTES = SCALE_BUFS * (int)sizeof(ScaleChunk<BN2>);
constexpr int SMEM2_BASE = 1024 + STAGES2 * STAGE2_BYTES + EPI_WARPS * OUT_WARP + SCALE2_BYTES + 256;
// Biases of three tiles: the scales' warp, which fetches them, may be two tiles
// ahead of the warps that still store one.
constexpr int BIAS_BUFS = 3;
constexpr int BIAS_BYTES = BIAS_BUFS * BN2 * 4;
constexpr int RES_BYTES = EPI_WARPS * OUT_WARP;  // two buffers like a warp's for its results
static_assert(RES_BYTES <= STAGE2_BYTES, "in the place of a stage");

// What the tiles cover.
constexpr int WALK_WHOLE = 0;  // one matrix
constexpr int WALK_ROWS = 1;   // rows of A and C in groups with a B each
constexpr int WALK_BLOCKS = 2; // columns of A and B in groups with a C each
// What happens to the sums: stored as they are, or an epilogue whose activation is
// none, relu or one of the others' RG_ACT_*.  An instance for each of these: the
// code of an activation stands 128 times in the loop over a warp's columns.
constexpr int PLAIN = -1;
constexpr int SIMPLE_ACT = RG_ACT_NONE;
__host__ __device__ constexpr int pair_smem(int walk, int act) {
  return SMEM2_BASE + (walk != WALK_WHOLE ? (int)sizeof(GroupTable) : 0) + (act != PLAIN ? BIAS_BYTES : 0);
}
static_assert(pair_smem(WALK_ROWS, PLAIN) <= 232448 && pair_smem(WALK_WHOLE, SIMPLE_ACT) <= 232448, "shared memory");

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

// Tile t of a CTA pair: rows [m0, m_end) of A from m0 on, columns from n0 on,
// blocks [kb0, kb1), matrix g.  Tiles of one matrix run down its rows first.
struct TileAt {
  int m0, m_end, n0, kb0, kb1, g;
};
template <int WALK>
struct Walk {
  const Params& gp;
  const GroupTable& tab;
  int g = 0;
  // t grows from call to call
  __device__ __forceinline__ TileAt at(int t) {
    if constexpr (WALK == WALK_WHOLE) {
      const int tn = t / gp.mt, tm = t - tn * gp.mt;
      return TileAt{tm * 256, gp.M, tn * BN2, 0, gp.KB, 0};
    } else if constexpr (WALK == WALK_ROWS) {
      while (t >= tab.first[g + 1]) ++g;
      const int row = tab.rows[g], end = tab.rows[g + 1], mt = (end - row + 255) / 256, i = t - tab.first[g];
      const int tn = i / mt, tm = i - tn * mt;
      return TileAt{row + tm * 256, end, tn * BN2, 0, g < gp.gr.E ? gp.KB : 0, g};
    } else {
      const int tiles = gp.mt * gp.nt;
      g = t / tiles;
      const int i = t - g * tiles, tn = i / gp.mt, tm = i - tn * gp.mt;
      const int kb0 = first_block(tab.rows[g], g);
      return TileAt{tm * 256, gp.M, tn * BN2, kb0, kb0 + (tab.rows[g + 1] - tab.rows[g] + 127) / 128, g};
    }
  }
};

// Byte `at` of row r's 64 in a staging buffer, whose 16-byte chunks are swizzled as
// the TMA's 64-byte mode has them.
__device__ __forceinline__ uint32_t staged(int r, int at) {
  return r * 64 + (((at >> 4) ^ ((r >> 1) & 3)) << 4) + (at & 15);
}
// The largest unit (up to `unit`) of which `bytes` is a multiple.
__device__ __forceinline__ int unit_of(int unit, int bytes) {
  while (bytes & (unit - 1)) unit >>= 1;
  return unit;
}
// Rows of `bytes` (up to 64) from a staging buffer to memory, `pitch` bytes apart, a
// unit to a lane: neighbouring lanes write neighbouring units.
template <typename Unit>
__device__ __forceinline__ void store_units(uint8_t* out, long long pitch, const uint8_t* buf, int rows, int bytes,
                                            int lane) {
  constexpr int PER = 64 / sizeof(Unit);  // lanes to a row
  const int at = (lane % PER) * (int)sizeof(Unit);
  if (at < bytes) {
#pragma unroll 4
    for (int r = lane / PER; r < rows; r += 32 / PER)
      *reinterpret_cast<Unit*>(out + r * pitch + at) = *reinterpret_cast<const Unit*>(buf + staged(r, at));
  }
}
__device__ __forceinline__ void store_units(uint8_t* out, long long pitch, const uint8_t* buf, int rows, int bytes,
                                            int u, int lane) {
  if (u == 16) store_units<uint4>(out, pitch, buf, rows, bytes, lane);
  else if (u == 8) store_units<uint2>(out, pitch, buf, rows, bytes, lane);
  else if (u == 4) store_units<uint32_t>(out, pitch, buf, rows, bytes, lane);
  else store_units<uint16_t>(out, pitch, buf, rows, bytes, lane);
}
// The same as a call, for the kernels with an epilogue, whose unrolled loops over
// columns would hold many copies (8192 x 4092 x 2048 with a bias 108 us, 85 called; in
// the kernels without, calls cost 5 to 10%).
__device__ __noinline__ void store_ragged(uint8_t* out, long long pitch, const uint8_t* buf, int rows, int bytes,
                                          int u, int lane) {
  store_units(out, pitch, buf, rows, bytes, u, lane);
}
// 64 bytes of each of a warp's rows leave its staging buffer for columns cc.. of D.
// Where D's rows start on 16-byte boundaries and all 32 rows are the tile's, a TMA
// store takes them away and cuts them to the matrix; else the warp writes them, in
// the largest units that fit (8192 x 4096 x 2048 bf16: 65 us; of 4092 columns 75, 4094
// 79, 4095 90.  Entry by entry, two to a lane: 91 each.  The unit found anew at each
// row: 86, 109 and 143).
template <int ES, bool CALL = false>
__device__ __forceinline__ void store_chunk(const CUtensorMap* tm, bool tma, void* D, long long ldd, int unit,
                                            const uint8_t* buf, int row0, int rows, int cc, int N, int lane) {
  constexpr int COLS = 64 / ES;
  if (tma) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (cc < N)
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(tm)),
                     "r"(smem_u32(buf)), "r"(cc), "r"(row0)
                     : "memory");
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  const int bytes = min(COLS, N - cc) * ES;
  if (bytes > 0) {
    uint8_t* out = static_cast<uint8_t*>(D) + ((long long)row0 * ldd + cc) * ES;
    const long long pitch = ldd * ES;
    const int u = unit_of(unit, bytes);
    if constexpr (CALL) store_ragged(out, pitch, buf, rows, bytes, u, lane);
    else store_units(out, pitch, buf, rows, bytes, u, lane);
  }
  __syncwarp();
}
// The staging buffer that the last store but one used has been read.
__device__ __forceinline__ void buffer_free(bool tma, int lane) {
  if (tma) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
  }
}
// Two neighbouring entries in C's type.
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
// 64 bytes of a row's sums (a row to a lane), 16 bytes at a time.
template <int ES>
__device__ __forceinline__ void stage_row(uint8_t* buf, const uint64_t* acc, int type, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 w;
    if constexpr (ES == 4) {
      const float2 f = unpack2(acc[2 * i]), h = unpack2(acc[2 * i + 1]);
      w = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(h.x), __float_as_uint(h.y));
    } else {
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = packed<ES>(unpack2(acc[4 * i + j]), type);
      w = make_uint4(p[0], p[1], p[2], p[3]);
    }
    *reinterpret_cast<uint4*>(buf + staged(lane, 16 * i)) = w;
  }
}

// This warp's 32 rows x 128 columns of sums to C through two alternating staging
// buffers.  c_row0: row0 in C, whose matrices may lie one behind the other.  (Four
// buffers in a stage's place were worth 1% where little is summed for much that is
// stored, in sums over groups.)
template <int ES, bool TILE_B, int WALK>
__device__ __forceinline__ void store_rows(const Params& gp, const CUtensorMap* tmC,
                                           const Sums<PAIR_COLS, TILE_B>& sums, uint8_t* stage, int c_row0, int rows,
                                           int col0, int lane) {
  constexpr int COLS = 64 / ES;
  // a whole matrix's last rows are cut by the TMA store too
  const bool tma = gp.unit_c == 16 && (WALK == WALK_WHOLE || rows == 32);
  if (WALK != WALK_WHOLE && gp.unit_c == 16 && !tma) {  // the last tile's stores have read both buffers
    if (lane == 0) bulk_wait_read0();
    __syncwarp();
  }
#pragma unroll
  for (int c = 0; c < PAIR_COLS / COLS; ++c) {
    uint8_t* buf = stage + (c & 1) * OUT_BUF;
    buffer_free(tma, lane);
    if constexpr (TILE_B) {
      stage_row<ES>(buf, sums.acc[0] + c * (COLS / 2), gp.out_type, lane);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (lane >> 2) + 8 * i;
#pragma unroll
        for (int j = 0; j < COLS / 8; ++j) {
          const int at = (8 * j + 2 * (lane & 3)) * ES;  // byte within the row's 64
          stage_pair<ES>(buf + staged(r, at), unpack2(sums.acc[i][c * (COLS / 8) + j]), gp.out_type);
        }
      }
    }
    store_chunk<ES>(tmC, tma, gp.C, gp.ldc, gp.unit_c, buf, c_row0, rows, col0 + c * COLS, gp.N, lane);
  }
}

// 64 bytes of each of a warp's rows of the residual, from column cc on, on their way
// to a buffer laid out like the ones for results, in the largest units that fit;
// units of two bytes, which no asynchronous copy takes, wait_residual fetches (8192 x
// 4096 x 2048 bf16: 81 us; of 4094 columns 121, 4095 156; each read where it is added: 477, 487).
template <typename Unit>
__device__ __forceinline__ void copy_units(uint32_t buf, const uint8_t* in, long long pitch, int rows, int bytes,
                                           int lane) {
  constexpr int PER = 64 / sizeof(Unit);  // lanes to a row
  const int at = (lane % PER) * (int)sizeof(Unit);
  if (at < bytes) {
#pragma unroll 4
    for (int r = lane / PER; r < rows; r += 32 / PER) {
      const uint32_t dst = buf + staged(r, at);
      const uint8_t* src = in + r * pitch + at;
      if constexpr (sizeof(Unit) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"((int)sizeof(Unit)) : "memory");
    }
  }
}
__device__ __noinline__ void copy_ragged(uint32_t buf, const uint8_t* in, long long pitch, int rows, int bytes, int u,
                                         int lane) {
  if (u == 16) copy_units<uint4>(buf, in, pitch, rows, bytes, lane);
  else if (u == 8) copy_units<uint2>(buf, in, pitch, rows, bytes, lane);
  else if (u == 4) copy_units<uint32_t>(buf, in, pitch, rows, bytes, lane);
}
// A lane to a column of two bytes, eight rows under way at a time.
__device__ __noinline__ void fetch_ragged(uint8_t* buf, const uint16_t* in, long long ld, int rows, int cols, int lane) {
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 8) {
    uint16_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r0 + i < rows && lane < cols ? in[(r0 + i) * ld] : (uint16_t)0;
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint16_t*>(buf + staged(r0 + i, 2 * lane)) = v[i];
  }
}
template <int ES, bool RAGGED>
__device__ __forceinline__ void start_residual(const Params& gp, uint8_t* buf, int row0, int rows, int cc, int lane) {
  const int bytes = min(64 / ES, gp.N - cc) * ES;
  if (bytes > 0) {
    const uint8_t* in = static_cast<const uint8_t*>(gp.ep.R) + ((long long)row0 * gp.ep.ldr + cc) * ES;
    const long long pitch = gp.ep.ldr * ES;
    if constexpr (RAGGED) copy_ragged(smem_u32(buf), in, pitch, rows, bytes, unit_of(gp.unit_r, bytes), lane);
    else copy_units<uint4>(smem_u32(buf), in, pitch, rows, bytes, lane);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int ES, bool RAGGED>
__device__ __forceinline__ void wait_residual(const Params& gp, uint8_t* buf, int row0, int rows, int cc, int lane) {
  asm volatile("cp.async.wait_group 1;" ::: "memory");  // all but the next chunk's
  if constexpr (RAGGED && ES == 2) {
    const int cols = min(32, gp.N - cc);
    if (cols > 0 && unit_of(gp.unit_r, cols * 2) == 2) {
      const uint16_t* in = static_cast<const uint16_t*>(gp.ep.R) + (long long)row0 * gp.ep.ldr + cc + lane;
      fetch_ragged(buf, in, gp.ep.ldr, rows, cols, lane);
    }
  }
  __syncwarp();
}
template <int ES>
__device__ __forceinline__ float2 residual_pair(const uint4& r, int j, int type) {  // columns 2 j, 2 j + 1 of 16 bytes
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  if constexpr (ES == 4) return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  else if (type == RG_TYPE_F16) return __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
  else return make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
}

// The same with an epilogue: sums + bias, stored where they are wanted before the
// activation, then the activation and the residual.  The residual comes 64 bytes
// of each row at a time through a ring of two buffers, the first two of them since
// the tile began (start_residual there).
template <int ES, int ACT, bool RES, bool RAGGED>
__device__ __forceinline__ void store_rows_act(const Params& gp, const CUtensorMap* tmC, const CUtensorMap* tmP,
                                               Sums<PAIR_COLS, true>& sums, const float* bias, uint8_t* stage,
                                               uint8_t* ring, int row0, int rows, int col0, int lane) {
  constexpr int COLS = 64 / ES, CHUNKS = PAIR_COLS / COLS, PER = 8 / ES;  // pairs of columns in 16 bytes
  const bool relu = ACT == SIMPLE_ACT && gp.ep.act == RG_ACT_RELU;
  const bool tma = !RAGGED || gp.unit_c == 16;
  int n = 0;  // stores
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    uint64_t* acc = sums.acc[0] + c * (COLS / 2);
    const int cc = col0 + c * COLS;
#pragma unroll
    for (int j = 0; j < COLS / 2; j += 2) {
      const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(bias + c * COLS + 2 * j);
      acc[j] = add2(acc[j], b.x);
      acc[j + 1] = add2(acc[j + 1], b.y);
    }
    if (gp.ep.P) {
      buffer_free(tma, lane);
      uint8_t* buf = stage + (n++ & 1) * OUT_BUF;
      stage_row<ES>(buf, acc, gp.out_type, lane);
      store_chunk<ES, RAGGED>(tmP, tma, gp.ep.P, gp.ldc, gp.unit_c, buf, row0, rows, cc, gp.N, lane);
    }
    uint8_t* in = ring + (c & 1) * OUT_BUF;
    if constexpr (RES) wait_residual<ES, RAGGED>(gp, in, row0, rows, cc, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 res = make_uint4(0, 0, 0, 0);
      if constexpr (RES) res = *reinterpret_cast<const uint4*>(in + staged(lane, 16 * i));
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        uint64_t& a = acc[i * PER + j];
        const float2 f = unpack2(a);
        if constexpr (ACT == SIMPLE_ACT) {
          if (relu) a = pack2(activate<RG_ACT_RELU>(f.x), activate<RG_ACT_RELU>(f.y));
        } else {
          a = pack2(activate<ACT>(f.x), activate<ACT>(f.y));
        }
        if constexpr (RES) {
          const float2 r = residual_pair<ES>(res, j, gp.out_type);
          a = add2(a, pack2(r.x, r.y));
        }
      }
    }
    if constexpr (RES) {
      __syncwarp();
      if (c + 2 < CHUNKS) start_residual<ES, RAGGED>(gp, in, row0, rows, cc + 2 * COLS, lane);
      else asm volatile("cp.async.commit_group;" ::: "memory");
    }
    buffer_free(tma, lane);
    uint8_t* buf = stage + (n++ & 1) * OUT_BUF;
    stage_row<ES>(buf, acc, gp.out_type, lane);
    store_chunk<ES, RAGGED>(tmC, tma, gp.C, gp.ldc, gp.unit_c, buf, row0, rows, cc, gp.N, lane);
  }
}

// RAGGED, with an epilogue: rows of C or of the residual that start or end off a
// 16-byte boundary.  Instances of their own: those that can do both took 74 us for 8192
// x 4096 x 2048 bf16 with a bias, 90 with a residual, 112 with these, silu and stored
// values; without the other path 71, 81 and 96.
template <bool B_KMAJOR, bool TILE_B, int WALK, int ACT, bool RES, bool RAGGED>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    f8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmP,
                        const __grid_constant__ Params gp, DevPlan* plan) {
  static_assert(ACT == PLAIN ? !RES : TILE_B && WALK == WALK_WHOLE, "an epilogue has a row to a lane");
  static_assert(ACT != PLAIN || !RAGGED, "found out as it runs");
  constexpr int STAGES = RES ? STAGES2_RING : STAGES2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t rank = cluster_rank();
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stage_base = smem;
  uint8_t* out_base = smem + STAGES2 * STAGE2_BYTES;
  uint8_t* ring_base = smem + STAGES2_RING * STAGE2_BYTES;  // RES
  ScaleChunk<BN2>* scales = reinterpret_cast<ScaleChunk<BN2>*>(out_base + EPI_WARPS * OUT_WARP);
  uint64_t* bars = reinterpret_cast<uint64_t*>(out_base + EPI_WARPS * OUT_WARP + SCALE2_BYTES);
  uint8_t* more = reinterpret_cast<uint8_t*>(bars) + 256;
  GroupTable& tab = *reinterpret_cast<GroupTable*>(more);   // WALK_ROWS, WALK_BLOCKS
  float* bias_base = reinterpret_cast<float*>(more);        // epilogues
  uint64_t* full = bars;
  uint64_t* done = bars + STAGES;         // by half * STAGES + stage: the half's MMAs of the stage are complete
  uint64_t* tempty = bars + 3 * STAGES;  // by half * 2 + accumulator
  uint64_t* sfull = tempty + 4;
  uint64_t* sempty = sfull + SCALE_BUFS;
  uint64_t* drain = sempty + SCALE_BUFS;  // by half
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ctl ctl{abort_flag, &plan->status, &plan->timeout_where, gp.wait_ns};

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&done[s]), 1);
      mbar_init(smem_u32(&done[STAGES + s]), 1);
    }
    for (int b = 0; b < 4; ++b) mbar_init(smem_u32(&tempty[b]), EPI_WARPS);  // the half's warps of both CTAs
    for (int b = 0; b < SCALE_BUFS; ++b) {
      mbar_init(smem_u32(&sfull[b]), ACT == PLAIN ? 32 : 33);  // 33: the bias
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
  if (!gp.late) wait_for_predecessor();
  start_status(gp, plan);
  int total = gp.mt * gp.nt;
  if constexpr (WALK == WALK_ROWS) total = load_groups(gp.gr, tab, 256, gp.nt, plan);
  if constexpr (WALK == WALK_BLOCKS) total *= load_groups(gp.gr, tab, 0, 0, plan) * gp.gr.E;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      Walk<WALK> walk{gp, tab};
      for (int t = cid; t < total && ok; t += ncl) {
        const TileAt at = walk.at(t);
        for (int kb = at.kb0; kb < at.kb1; ++kb) {
          if (!wait_bounded(smem_u32(&done[stage]), phase ^ 1u, ctl, 31) ||
              !wait_bounded(smem_u32(&done[STAGES + stage]), phase ^ 1u, ctl, 31)) {
            ok = false;
            break;
          }
          const uint32_t fb_local = smem_u32(&full[stage]);
          if (rank == 0) mbar_arrive_expect_tx(fb_local, 2 * STAGE2_BYTES);
          const uint32_t fb = mapa_shared(fb_local, 0);
          const uint32_t a_dst = smem_u32(stage_base + stage * STAGE2_BYTES);
          tma_load_2d_pair(a_dst, &tmA, fb, kb * BK, at.m0 + (int)rank * 128);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t b_dst = a_dst + SLAB + h * HALF_SLAB;
            const int n0 = at.n0 + h * 128 + (int)rank * 64;
            if constexpr (WALK == WALK_ROWS) {
              if constexpr (B_KMAJOR) tma_load_3d_pair(b_dst, &tmB, fb, kb * BK, n0, at.g);
              else tma_load_3d_pair(b_dst, &tmB, fb, n0, kb * BK, at.g);
            } else {
              if constexpr (B_KMAJOR) tma_load_2d_pair(b_dst, &tmB, fb, kb * BK, n0);
              else tma_load_2d_pair(b_dst, &tmB, fb, n0, kb * BK);
            }
          }
          if (++stage == STAGES) {
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
      Walk<WALK> walk{gp, tab};
      for (int t = cid; t < total && ok; t += ncl) {
        const TileAt at = walk.at(t);
        for (int kb = at.kb0; kb < at.kb1; ++kb, ++it) {
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
            if (!(gp.fault == 1 && it == 0)) umma_commit_pair(smem_u32(&done[half * STAGES + stage]));
          }
          __syncwarp();
          if (++stage == STAGES) {
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
      Walk<WALK> walk{gp, tab};
      int slot = 0;  // of the biases
      for (int t = cid; t < total && ok; t += ncl) {
        const TileAt at = walk.at(t);
        const float* SB = WALK == WALK_ROWS ? gp.SB + at.g * gp.sb_e : gp.SB;
        for (int kb = at.kb0; kb < at.kb1 && ok; kb += KC, ++c) {
          const int b = c & 1;
          ok = wait_bounded(smem_u32(&sempty[b]), ((c >> 1) & 1u) ^ 1u, ctl, 35);
          if (!ok) break;
          load_scales<BN2, TILE_B, 32>(gp, SB, scales[b], at.m0 + (int)rank * 128, at.n0, kb, at.kb1, lane);
          if constexpr (ACT != PLAIN) {
            if (kb == at.kb0) {
              float* bias = bias_base + slot * BN2;
              for (int j = lane; j < BN2; j += 32)
                bias[j] = gp.ep.bias && at.n0 + j < gp.N ? load_real(gp.ep.bias, gp.ep.bias_type, at.n0 + j) : 0.0f;
              slot = slot + 1 == BIAS_BUFS ? 0 : slot + 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sfull[b]));
          }
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
    Walk<WALK> walk{gp, tab};
    int slot = 0;  // of the biases
    for (int t = cid; t < total && ok; t += ncl) {
      const TileAt at = walk.at(t);
      const int row0 = at.m0 + (int)rank * 128 + q4 * 32, col0 = at.n0 + col;
      // a group's last tile: warps without a row of it leave the sums alone
      const bool mine = WALK != WALK_ROWS || row0 < at.m_end;
      uint8_t* ring = ring_base + ew * OUT_WARP;
      if constexpr (RES) {
        const int rows = min(32, at.m_end - row0), es = gp.out_type == RG_TYPE_F32 ? 4 : 2;
        for (int c = 0; c < 2; ++c) {
          uint8_t* buf = ring + c * OUT_BUF;
          if (es == 4) start_residual<4, RAGGED>(gp, buf, row0, rows, col0 + c * 16, lane);
          else start_residual<2, RAGGED>(gp, buf, row0, rows, col0 + c * 32, lane);
        }
        // the rest of the warp's rows, as far as L2
        if (lane < rows && col0 < gp.N) {
          const uint8_t* p = static_cast<const uint8_t*>(gp.ep.R) + ((long long)(row0 + lane) * gp.ep.ldr + col0) * es;
          const int bytes = min(PAIR_COLS, gp.N - col0) * es;
          for (int i = RAGGED ? 0 : 128; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
        }
      }
      using Acc = Sums<PAIR_COLS, TILE_B>;
      Acc sums = {};
      for (int kb = at.kb0; kb < at.kb1; ++kb, ++it) {
        const uint32_t b = it & 1u;
        const int kbi = (kb - at.kb0) % KC;
        const ScaleChunk<BN2>& sc = scales[chunk & 1];
        ok = kbi != 0 || wait_bounded(smem_u32(&sfull[chunk & 1]), (chunk >> 1) & 1u, ctl, 36);
        ok = __all_sync(0xFFFFFFFFu, ok && wait_bounded(smem_u32(&done[half * STAGES + st]), phase, ctl, 34));
        if (++st == STAGES) {
          st = 0;
          phase ^= 1u;
        }
        if (!ok) break;
        tc_fence_after();
        auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed_cluster(tempty_leader[b]);
        };
        if (mine) {
          float s[Acc::kRows];
#pragma unroll
          for (int i = 0; i < Acc::kRows; ++i) {
            s[i] = sc.a[kbi][q4 * 32 + Acc::row(lane, i)];
            if constexpr (TILE_B) s[i] *= sc.b[kbi][half];
          }
          sums.add(lane_addr + b * 128, s, &sc.b[kbi][col], release);
        } else {
          release();
        }
        if (kbi == KC - 1 || kb == at.kb1 - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sempty[chunk & 1]));
          ++chunk;
        }
      }
      if constexpr (WALK == WALK_BLOCKS) {
        // found again: kept over the blocks' loop, where no register is free, they spilled
        int u = t;
        asm volatile("" : "+r"(u));
        const TileAt at2 = walk.at(u);
        const int row = at2.m0 + (int)rank * 128 + q4 * 32, n0 = at2.n0 + col;
        if (ok && row < gp.M && n0 < gp.N) {
          const int rows = min(32, gp.M - row), c_row = row + at2.g * gp.M;
          if (gp.out_type == RG_TYPE_F32) store_rows<4, TILE_B, WALK>(gp, &tmC, sums, stage, c_row, rows, n0, lane);
          else store_rows<2, TILE_B, WALK>(gp, &tmC, sums, stage, c_row, rows, n0, lane);
        }
      } else if (ok && row0 < at.m_end && col0 < gp.N) {
        const int rows = min(32, at.m_end - row0);
        if constexpr (ACT != PLAIN) {
          // nothing that is computed from these before the blocks' loop
          int r0 = row0, c0 = col0, l = lane;
          asm volatile("" : "+r"(r0), "+r"(c0), "+r"(l));
          const float* bias = bias_base + slot * BN2 + (ew >> 2) * PAIR_COLS;
          if (gp.out_type == RG_TYPE_F32)
            store_rows_act<4, ACT, RES, RAGGED>(gp, &tmC, &tmP, sums, bias, stage, ring, r0, rows, c0, l);
          else
            store_rows_act<2, ACT, RES, RAGGED>(gp, &tmC, &tmP, sums, bias, stage, ring, r0, rows, c0, l);
        } else {
          if (gp.out_type == RG_TYPE_F32)
            store_rows<4, TILE_B, WALK>(gp, &tmC, sums, stage, row0, rows, col0, lane);
          else
            store_rows<2, TILE_B, WALK>(gp, &tmC, sums, stage, row0, rows, col0, lane);
        }
      }
      if constexpr (ACT != PLAIN) slot = slot + 1 == BIAS_BUFS ? 0 : slot + 1;
    }
    if constexpr (RES) asm volatile("cp.async.wait_all;" ::: "memory");
    bulk_wait0();
  }

  __syncwarp();  // whole warps again before the abort check and the barriers below
  if (gp.late) wait_for_predecessor();
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

using PairKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const Params,
                            DevPlan*);

template <bool RAGGED>
const void* pair_act_instance(int act, bool residual) {
  auto pick = [residual](PairKernel with, PairKernel without) {
    return reinterpret_cast<const void*>(residual ? with : without);
  };
#define RG_PAIR_ACT(ACT) \
  pick(f8_gemm_pair_kernel<true, true, WALK_WHOLE, ACT, true, RAGGED>, \
       f8_gemm_pair_kernel<true, true, WALK_WHOLE, ACT, false, RAGGED>)
  switch (act) {
    case RG_ACT_SILU: return RG_PAIR_ACT(RG_ACT_SILU);
    case RG_ACT_GELU: return RG_PAIR_ACT(RG_ACT_GELU);
    case RG_ACT_GELU_TANH: return RG_PAIR_ACT(RG_ACT_GELU_TANH);
    default: return RG_PAIR_ACT(SIMPLE_ACT);
  }
#undef RG_PAIR_ACT
}

// The maps of A, of C and of what an epilogue stores before the activation.
bool pair_maps(const F8GemmArgs& a, const Params& p, int dev, CUtensorMap* ma, CUtensorMap* mc, CUtensorMap* mp,
               long long c_rows) {
  const int es = a.out_type == RG_TYPE_F32 ? 4 : 2;
  const CUtensorMapDataType type = es == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  auto out_map = [&](CUtensorMap* m, const void* base) {
    return make_map_2d(m, dev, base, (uint64_t)a.N, (uint64_t)c_rows, (uint64_t)a.ldc * es, 64 / es, 32,
                       CU_TENSOR_MAP_SWIZZLE_64B, type);
  };
  return make_map_2d(ma, dev, a.A, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.lda, BK, 128) &&
         (p.unit_c != 16 || (out_map(mc, a.C) && (!p.ep.P || out_map(mp, p.ep.P))));
}

}  // namespace
}  // namespace rg
