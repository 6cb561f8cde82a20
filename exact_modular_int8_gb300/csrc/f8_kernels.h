// f8_kernels.h -- launchers of the 8-bit block-scaled kernels (internal, C++ linkage).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "rg_common.cuh"

namespace rg {

// The largest of 16, 8, 4 and 2 bytes on whose boundaries all rows start.
inline int row_unit(const void* p, long long row_bytes) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p) | (uintptr_t)row_bytes;
  return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
}

// X [M][K] (row stride ldx, in entries) to E4M3: Q [M][ldq] with S
// [M][ceil(K/128)] (rows) or [ceil(M/128)][ceil(K/128)] (tiles), and / or its
// transpose QT [K][ldqt] with ST [K][ceil(M/128)] (columns).
struct QuantArgs {
  const void* X;
  long long ldx, M, K;
  uint8_t* Q;
  long long ldq;
  float* S;
  uint8_t* QT;
  long long ldqt;
  float* ST;
  int unit_x, unit_p;     // set by the launcher: rows start on boundaries of 16, 8, 4 or 2 bytes
  bool vec_q, vec_qt;     // and on 8 and 16
  // tiles: this many matrices, M rows apart
  long long batch = 1;
  // columns, both: rows in groups (F8Groups), QT [K][128 blocks], ST [K][blocks]
  const void* offsets = nullptr;
  int wide = 0, E = 0;
  long long* kept_offsets = nullptr;  // a copy of them, [E + 1]
  long long blocks = 0;
  // both: X times the slope of the activation act at P [M][K] (X's type)
  int act = RG_ACT_NONE;
  const void* P = nullptr;
  // both: sums over the rows, [K] in out_type to `out` where kSumCluster blocks of 128
  // rows hold them all, else over each such block's, [ceil(M/128)][K], to `sums`
  float* sums = nullptr;
  void* out = nullptr;
  int out_type = RG_TYPE_F32;
  bool late = false;  // tiles: see F8GemmArgs
};
constexpr int kSumCluster = 8;
cudaError_t launch_quantise_f8(QuantArgs a, int type, int form, cudaStream_t st);
// out [K] = the sum of `rows` rows of partial sums [rows][K], in a fixed order.
cudaError_t launch_sum_rows(const float* sums, long long rows, long long K, void* out, int type, cudaStream_t st);

// What happens to a product's sums p before they are stored: p + bias[n] goes to P
// (C's type and row stride) where that is given, act(p + bias[n]) + R[m][n] to C.
struct F8Epilogue {
  const void* bias = nullptr;  // [N]
  int bias_type = RG_TYPE_F32;
  int act = RG_ACT_NONE;
  const void* R = nullptr;  // [M][ldr], C's type
  long long ldr = 0;
  void* P = nullptr;
};

// C [M][N] = sum over 128-blocks kb of sa[m][kb] sb[n][kb] (A_kb B_kb^T).
// A [M][lda] E4M3, K contiguous.  B [N][ldb] (b_kmajor) or [K][ldb] E4M3.
// SA is contiguous [M][KB], KB = ceil(K/128); the scale of B's column n in
// block kb is SB[(tile_b ? n / 128 : n) * sb_n + kb * sb_k].
struct F8GemmArgs {
  const uint8_t* A;
  const uint8_t* B;
  const float* SA;
  const float* SB;
  void* C;
  long long lda, ldb, ldc, sb_n, sb_k;
  long long M, N, K;
  int out_type;  // RG_TYPE_*
  bool b_kmajor, tile_b;
  bool keep_status = false;  // an earlier product of the same call has cleared it
  const F8Epilogue* ep = nullptr;  // b_kmajor and tile_b only
  // Reads nothing that the kernel before it in the stream writes, nor writes what
  // that reads, so that the two may run at the same time: it waits for that kernel
  // as it ends, not as it starts.  What the kernels further back wrote is there: the
  // one before has waited for them before it let this one start, or is late itself
  // and was let by one that had.  (A call's first kernel is never late.)
  bool late = false;
};
cudaError_t launch_f8_gemm(const F8GemmArgs& a, DevPlan* plan, cudaStream_t st, int fault,
                           unsigned long long wait_ns);

// The pair kernel with an epilogue (f8_act.cu, f8_act_ragged.cu); its parameters are those of f8_gemm.cu's.
const void* pair_act_kernel(int act, bool residual);
const void* pair_act_ragged_kernel(int act, bool residual);

// Products by group, group g holding rows (or, by_blocks, columns along the
// contraction) offsets[g] .. offsets[g + 1].
//   rows    C [M][N]: rows of group g times B[g], where B [E][N][ldb] (b_kmajor) or
//           [E][K][ldb], sb_e scales apart, in tiles
//   blocks  C [E][M][N]: the sum over group g's blocks of 128 columns of A [M][lda]
//           and B [N][ldb], which start at block offsets[g] / 128 + g; SA and SB are
//           [M][blocks], [N][blocks], K = 128 blocks; C's matrices lie without gaps
struct F8Groups {
  const void* offsets;  // [E + 1], device
  bool wide;            // 64-bit
  long long E;
  bool zero_rest;  // rows: write 0 to the rows behind the last group
  bool by_blocks;
  long long rows;  // offsets end here at the latest
};
cudaError_t launch_f8_grouped(const F8GemmArgs& a, const F8Groups& g, DevPlan* plan, cudaStream_t st, int fault,
                              unsigned long long wait_ns);

// The same for M <= kSkinnyRows and a transposed B.
constexpr int kSkinnyRows = 32;
cudaError_t launch_f8_skinny(const F8GemmArgs& a, DevPlan* plan, cudaStream_t st);

// Mixture-of-experts layer of T <= RG_MOE_MAX_TOKENS tokens (moe_layer_f8).
struct MoeArgs {
  const void* X;        // [T][H]
  const void* WR;       // [E][H]
  const uint8_t* W13;   // [E][2I][H]
  const float* S13;     // [E][ceil(2I/128)][ceil(H/128)]
  const uint8_t* W2;    // [E][H][I]
  const float* S2;      // [E][ceil(H/128)][ceil(I/128)]
  void* Y;              // [T][H]
  long long T, H, I, E, top_k;
  int type;  // of X, WR and Y: RG_TYPE_F16 or RG_TYPE_BF16
  bool renorm;
};
size_t moe_f8_scratch_bytes(long long T, long long H, long long I, long long top_k);
cudaError_t launch_moe_f8(const MoeArgs& a, DevPlan* plan, void* scratch, cudaStream_t st,
                          unsigned long long wait_ns);

}  // namespace rg
