// f8_api.cu -- the C ABI of the 8-bit block-scaled operators (include/resgemm.h):
// validation, then one launcher each.
#include <climits>
#include <cstdint>

#include "f8_kernels.h"
#include "rg_call.h"
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

// C = A B (an empty sum where K is 0) for operands that have been checked;
// the kernels clear the status themselves.
int product(const F8GemmArgs& a, DevPlan* plan, cudaStream_t st) {
  const size_t es = a.out_type == RG_TYPE_F32 ? 4 : 2;
  if (!(a.M && a.N && a.K)) {
    if (!a.keep_status && cudaMemsetAsync(plan, 0, sizeof(DevPlan), st) != cudaSuccess) return RG_ERR_CUDA;
    if (a.M && a.N && cudaMemset2DAsync(a.C, (size_t)a.ldc * es, 0, (size_t)a.N * es, (size_t)a.M, st) != cudaSuccess)
      return RG_ERR_CUDA;
    return RG_OK;
  }
  return launch_f8_gemm(a, plan, st, take_fault(), wait_limit_ns()) == cudaSuccess ? RG_OK : RG_ERR_CUDA;
}

int quantise(const QuantArgs& a, int type, int form, cudaStream_t st) {
  if (!a.M || !a.K) return RG_OK;
  return launch_quantise_f8(a, type, form, st) == cudaSuccess ? RG_OK : RG_ERR_CUDA;
}

// Scales of a contiguous B operand as scaled_gemm_f8 lays them out.
F8GemmArgs gemm_args(const uint8_t* A, long long lda, const float* SA, const uint8_t* B, long long ldb, const float* SB,
                     void* C, int c_type, long long ldc, long long M, long long N, long long K, bool transb,
                     bool tile_b) {
  const long long kb = blocks128(K), nb = tile_b ? blocks128(N) : N;
  return F8GemmArgs{A, B, SA, SB, C, lda, ldb, ldc, transb ? kb : 1, transb ? 1 : nb, M, N, K, c_type, transb, tile_b};
}

// Consecutive 256-byte aligned pieces of a buffer (null: sizes only).
struct Carver {
  uint8_t* base;
  size_t off = 0;
  uint8_t* take(size_t bytes) {
    uint8_t* p = base ? base + off : nullptr;
    off += (bytes + 255) & ~size_t(255);
    return p;
  }
};
// A quantised matrix of `rows` x `cols`: values with rows on 16-byte boundaries, and scales.
struct Quantised {
  uint8_t* q;
  float* s;
  long long ld;
};
Quantised carve(Carver& c, long long rows, long long cols, long long scale_rows) {
  Quantised m;
  m.ld = (cols + 15) & ~15LL;
  m.q = c.take((size_t)rows * m.ld);
  m.s = reinterpret_cast<float*>(c.take((size_t)scale_rows * blocks128(cols) * 4));
  return m;
}
// What a linear layer's forward pass keeps: X^T and the weights.
struct Saved {
  Quantised xt, w;
  size_t bytes;
};
Saved carve_saved(uint8_t* base, long long M, long long N, long long K) {
  Carver c{base};
  Saved v;
  v.xt = carve(c, K, M, K);
  v.w = carve(c, N, K, blocks128(N));
  v.bytes = c.off;
  return v;
}
bool good_linear(long long M, long long N, long long K) {
  return M >= 0 && N >= 0 && K >= 0 && M <= kMaxDim && N <= kMaxDim && K <= kMaxDim &&
         blocks128(M) * blocks128(N) <= INT_MAX / 8 && blocks128(M) * blocks128(K) <= INT_MAX / 8 &&
         blocks128(N) * blocks128(K) <= INT_MAX / 8;
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
    const int rc = quantise(QuantArgs{X, ldx, M, K, Q, ldq, S, QT, ldqt, ST, false, false, false}, x_type, form, st);
    if (rc) return rc;
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
  DevPlan* plan = static_cast<DevPlan*>(ws);
  if (M && N && (!C || ldc < N)) return RG_ERR_ARG;
  if (M && N && K) {
    if (!A || !B || !SA || !SB || lda < K || ldb < (transb ? K : N) || !aligned16(A, lda) || !aligned16(B, ldb))
      return RG_ERR_ARG;
    if (blocks128(M) * blocks128(N) > INT_MAX / 8) return RG_ERR_ARG;
  }
  const WorkspaceTurn turn(ws);
  const int rc = product(gemm_args(A, lda, SA, B, ldb, SB, C, c_type, ldc, M, N, K, transb, tile_b), plan, st);
  return rc ? rc : finish_call(ws, st, flags);
}

size_t linear_f8_saved_bytes(int64_t M, int64_t N, int64_t K) {
  return good_linear(M, N, K) ? carve_saved(nullptr, M, N, K).bytes + 256 : 0;
}

size_t linear_f8_ws_bytes(int64_t M, int64_t N, int64_t K) {
  if (!good_linear(M, N, K)) return 0;
  Carver forward{nullptr}, backward{nullptr};
  carve(forward, M, K, M);
  carve(backward, M, N, M);
  carve(backward, N, M, N);
  return kCallBlockBytes + (forward.off > backward.off ? forward.off : backward.off);
}

int linear_f8(const void* X, int x_type, int64_t ldx, const void* W, int w_type, int64_t ldw, void* Y, int64_t M,
              int64_t N, int64_t K, void* saved, size_t saved_bytes, unsigned flags, void* ws, size_t ws_bytes,
              void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || !saved || (reinterpret_cast<uintptr_t>(saved) & 255u) ||
      !good_type(x_type) || !good_type(w_type) || !good_linear(M, N, K))
    return RG_ERR_ARG;
  if (ws_bytes < linear_f8_ws_bytes(M, N, K) || saved_bytes < linear_f8_saved_bytes(M, N, K)) return RG_ERR_WORKSPACE;
  if ((M && K && (!X || ldx < K)) || (N && K && (!W || ldw < K)) || (M && N && !Y)) return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const Saved v = carve_saved(static_cast<uint8_t*>(saved), M, N, K);
  Carver c{static_cast<uint8_t*>(ws) + kCallBlockBytes};
  const Quantised x = carve(c, M, K, M);
  int rc = quantise(QuantArgs{X, ldx, M, K, x.q, x.ld, x.s, v.xt.q, v.xt.ld, v.xt.s, false, false, false}, x_type,
                    RG_F8_BOTH, st);
  if (!rc)
    rc = quantise(QuantArgs{W, ldw, N, K, v.w.q, v.w.ld, v.w.s, nullptr, 0, nullptr, false, false, false}, w_type,
                  RG_F8_TILES, st);
  if (!rc)
    rc = product(gemm_args(x.q, x.ld, x.s, v.w.q, v.w.ld, v.w.s, Y, x_type, N, M, N, K, true, true),
                 static_cast<DevPlan*>(ws), st);
  return rc ? rc : finish_call(ws, st, flags);
}

int linear_f8_backward(const void* dY, int dy_type, int64_t lddy, const void* saved, size_t saved_bytes, void* dX,
                       void* dW, int dw_type, int64_t M, int64_t N, int64_t K, unsigned flags, void* ws,
                       size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || !saved || (reinterpret_cast<uintptr_t>(saved) & 255u) ||
      !good_type(dy_type) || !good_type(dw_type) || !good_linear(M, N, K))
    return RG_ERR_ARG;
  if (ws_bytes < linear_f8_ws_bytes(M, N, K) || saved_bytes < linear_f8_saved_bytes(M, N, K)) return RG_ERR_WORKSPACE;
  if ((M && N && (!dY || lddy < N)) || (M && K && !dX) || (N && K && !dW)) return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const Saved v = carve_saved(static_cast<uint8_t*>(const_cast<void*>(saved)), M, N, K);
  DevPlan* plan = static_cast<DevPlan*>(ws);
  Carver c{static_cast<uint8_t*>(ws) + kCallBlockBytes};
  const Quantised d = carve(c, M, N, M), dt = carve(c, N, M, N);
  int rc = quantise(QuantArgs{dY, lddy, M, N, d.q, d.ld, d.s, dt.q, dt.ld, dt.s, false, false, false}, dy_type,
                    RG_F8_BOTH, st);
  if (!rc)  // dX [M][K] = dY [M][N] W [N][K]
    rc = product(gemm_args(d.q, d.ld, d.s, v.w.q, v.w.ld, v.w.s, dX, dy_type, K, M, K, N, false, true), plan, st);
  if (!rc) {  // dW [N][K] = dY^T [N][M] (X^T [K][M])^T
    F8GemmArgs a = gemm_args(dt.q, dt.ld, dt.s, v.xt.q, v.xt.ld, v.xt.s, dW, dw_type, K, N, K, M, true, false);
    a.keep_status = true;
    rc = product(a, plan, st);
  }
  return rc ? rc : finish_call(ws, st, flags);
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
  const WorkspaceTurn turn(ws);
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
