// f8_api.cu -- the C ABI of the 8-bit block-scaled operators (include/resgemm.h):
// validation, then one launcher each.
#include <climits>
#include <cstdint>

#include "f8_kernels.h"
#include "rg_kernels.h"

namespace {
using namespace rg;

constexpr long long kMaxDim = 1LL << 30;  // rows, columns and K: tile coordinates are 32-bit

bool good_type(int t) { return t == RG_TYPE_F32 || t == RG_TYPE_F16 || t == RG_TYPE_BF16; }
long long blocks128(long long x) { return (x + 127) / 128; }
bool aligned16(const void* p, long long row_bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (row_bytes & 15) == 0;
}

bool good_moe(long long T, long long H, long long I, long long E, long long top_k) {
  return T >= 0 && T <= RG_MOE_MAX_TOKENS && H >= 16 && I >= 16 && H % 16 == 0 && I % 16 == 0 &&
         H <= RG_MOE_MAX_WIDTH && I <= RG_MOE_MAX_WIDTH && E >= 1 && E <= RG_MOE_MAX_EXPERTS && top_k >= 1 &&
         top_k <= E && top_k <= RG_MOE_MAX_TOP_K;
}

}  // namespace

extern "C" {

int quantize_f8(const void* X, int x_type, int64_t ldx, int64_t M, int64_t K, int form, uint8_t* Q, int64_t ldq,
                float* S, uint8_t* QT, int64_t ldqt, float* ST, unsigned flags, void* stream) {
  if (!good_type(x_type) || form < RG_F8_ROWS || form > RG_F8_TILES || M < 0 || K < 0 || M > kMaxDim || K > kMaxDim)
    return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool direct = form != RG_F8_COLUMNS, transposed = form == RG_F8_COLUMNS || form == RG_F8_BOTH;
  if (M && K) {
    if (!X || ldx < K || (direct && (!Q || !S || ldq < K)) || (transposed && (!QT || !ST || ldqt < M)))
      return RG_ERR_ARG;
    const long long tiles = form == RG_F8_ROWS ? (M * blocks128(K) + 15) / 16 : blocks128(M) * blocks128(K);
    if (tiles > INT_MAX) return RG_ERR_ARG;
    QuantArgs a{X, ldx, M, K, Q, ldq, S, QT, ldqt, ST, false, false, false};
    if (launch_quantise_f8(a, x_type, form, st) != cudaSuccess) return RG_ERR_CUDA;
  }
  if ((flags & RG_FLAG_SYNC) && cudaStreamSynchronize(st) != cudaSuccess) return RG_ERR_CUDA;
  return RG_OK;
}

int scaled_gemm_f8(const uint8_t* A, int64_t lda, const float* SA, const uint8_t* B, int64_t ldb, const float* SB,
                   void* C, int c_type, int64_t ldc, int64_t M, int64_t N, int64_t K, unsigned flags, void* ws,
                   size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return RG_ERR_ARG;
  if (!good_type(c_type) || M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return RG_ERR_ARG;
  if (ws_bytes < kCallBlockBytes) return RG_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool transb = (flags & RG_FLAG_TRANS_B) != 0, tile_b = (flags & RG_FLAG_TILE_B) != 0;
  const size_t es = c_type == RG_TYPE_F32 ? 4 : 2;
  DevPlan* plan = static_cast<DevPlan*>(ws);
  if (M && N && (!C || ldc < N)) return RG_ERR_ARG;
  if (M && N && K) {
    if (!A || !B || !SA || !SB || lda < K || ldb < (transb ? K : N) || !aligned16(A, lda) || !aligned16(B, ldb))
      return RG_ERR_ARG;
    if (blocks128(M) * blocks128(N) > INT_MAX / 8) return RG_ERR_ARG;
  }
  if (!(M && N && K)) {  // an empty sum, or nothing at all (the kernels clear the status themselves)
    if (cudaMemsetAsync(plan, 0, sizeof(DevPlan), st) != cudaSuccess) return RG_ERR_CUDA;
    if (M && N && cudaMemset2DAsync(C, (size_t)ldc * es, 0, (size_t)N * es, (size_t)M, st) != cudaSuccess)
      return RG_ERR_CUDA;
  } else {
    const long long kb = blocks128(K), nb = tile_b ? blocks128(N) : N;
    F8GemmArgs a{A, B, SA, SB, C, lda, ldb, ldc, transb ? kb : 1, transb ? 1 : nb, M, N, K, c_type, transb, tile_b};
    if (launch_f8_gemm(a, plan, st, take_fault(), wait_limit_ns()) != cudaSuccess) return RG_ERR_CUDA;
  }
  return finish_call(ws, st, flags);
}

size_t moe_layer_f8_ws_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int top_k) {
  if (!good_moe(T, H, I, E, top_k)) return 0;
  return kCallBlockBytes + (T ? moe_f8_scratch_bytes(T, H, I, top_k) : 0);
}

int moe_layer_f8(const void* X, int x_type, const void* WR, const uint8_t* W13, const float* S13, const uint8_t* W2,
                 const float* S2, void* Y, int64_t T, int64_t H, int64_t I, int64_t E, int top_k, int renorm,
                 unsigned flags, void* ws, size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return RG_ERR_ARG;
  if ((x_type != RG_TYPE_F16 && x_type != RG_TYPE_BF16) || T < 0) return RG_ERR_ARG;
  if (T > RG_MOE_MAX_TOKENS) return RG_ERR_RANGE;
  if (!good_moe(T, H, I, E, top_k)) return RG_ERR_ARG;
  if (ws_bytes < moe_layer_f8_ws_bytes(T, H, I, E, top_k)) return RG_ERR_WORKSPACE;
  if (T && (!X || !WR || !W13 || !S13 || !W2 || !S2 || !Y || !aligned16(X, 0) || !aligned16(WR, 0) ||
            !aligned16(W13, 0) || !aligned16(W2, 0) || !aligned16(Y, 0)))
    return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T) {
    const MoeArgs a{X, WR, W13, S13, W2, S2, Y, T, H, I, E, top_k, x_type, renorm != 0};
    if (launch_moe_f8(a, static_cast<DevPlan*>(ws), static_cast<uint8_t*>(ws) + kCallBlockBytes, st,
                      wait_limit_ns()) != cudaSuccess)
      return RG_ERR_CUDA;
  } else if (cudaMemsetAsync(ws, 0, sizeof(DevPlan), st) != cudaSuccess) {
    return RG_ERR_CUDA;
  }
  return finish_call(ws, st, flags);
}

}  // extern "C"
