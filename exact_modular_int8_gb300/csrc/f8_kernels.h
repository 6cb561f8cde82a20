// f8_kernels.h -- launchers of the 8-bit block-scaled kernels (internal, C++ linkage).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "rg_common.cuh"

namespace rg {

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
  bool vec_x, vec_q, vec_qt;  // set by the launcher: rows start on 16 (8) byte boundaries
};
cudaError_t launch_quantise_f8(QuantArgs a, int type, int form, cudaStream_t st);

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
};
cudaError_t launch_f8_gemm(const F8GemmArgs& a, DevPlan* plan, cudaStream_t st, int fault,
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
