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

int reset_status(DevPlan* plan, cudaStream_t st) {
  return cudaMemsetAsync(plan, 0, sizeof(DevPlan), st) == cudaSuccess ? RG_OK : RG_ERR_CUDA;
}

// C = A B (an empty sum where K is 0) for operands that have been checked;
// the kernels clear the status themselves.
int product(const F8GemmArgs& a, DevPlan* plan, cudaStream_t st) {
  const size_t es = a.out_type == RG_TYPE_F32 ? 4 : 2;
  if (!(a.M && a.N && a.K)) {  // (with an epilogue K is at least 1)
    if (!a.keep_status && reset_status(plan, st)) return RG_ERR_CUDA;
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

// The gradients that a backward call computes, and the form in which they need the
// output's: along its rows for the input's, along its columns for the weights'.
struct Wanted {
  bool dx, dw;
  explicit Wanted(unsigned flags) : dx(!(flags & RG_FLAG_NO_DX)), dw(!(flags & RG_FLAG_NO_DW)) {}
  int form() const { return dx && dw ? RG_F8_BOTH : dx ? RG_F8_ROWS : RG_F8_COLUMNS; }
};

bool good_act(int act) { return act >= RG_ACT_NONE && act <= RG_ACT_GELU_TANH; }
size_t type_bytes(int t) { return t == RG_TYPE_F32 ? 4 : 2; }

// What a linear layer with an activation keeps: a linear layer's, and p.
struct SavedAct {
  Saved linear;
  uint8_t* p;
  size_t bytes;
};
SavedAct carve_saved_act(uint8_t* base, long long M, long long N, long long K, int x_type, int act) {
  SavedAct v;
  v.linear = carve_saved(base, M, N, K);
  Carver c{base, v.linear.bytes};
  v.p = act == RG_ACT_NONE ? nullptr : c.take((size_t)M * N * type_bytes(x_type));
  v.bytes = c.off;
  return v;
}

// Groups.
long long group_blocks(long long rows, long long E) { return rows / 128 + E; }
bool good_groups(long long rows, long long E, const void* offsets, unsigned flags) {
  return rows >= 0 && rows <= kMaxDim && E >= 1 && E <= RG_MOE_MAX_EXPERTS && offsets &&
         reinterpret_cast<uintptr_t>(offsets) % ((flags & RG_FLAG_OFFSETS64) ? 8 : 4) == 0;
}
bool good_expert_linear(long long T, long long N, long long K, long long E) {
  if (T < 0 || T > kMaxDim || N < 0 || N > kMaxDim || K < 1 || K > kMaxDim || E < 1 || E > RG_MOE_MAX_EXPERTS)
    return false;
  const long long tb = group_blocks(T, E) + 1, nb = blocks128(N), kb = blocks128(K);
  return tb * nb <= INT_MAX / 8 && tb * kb <= INT_MAX / 8 && E * nb * kb <= INT_MAX / 8 && E * N <= kMaxDim &&
         E * K <= kMaxDim;
}
struct SavedExperts {
  long long* offsets;  // [E + 1]
  Quantised xt, w;
  size_t bytes;
};
// A stack of `count` quantised matrices in tiles; a matrix's rows follow the last's.
Quantised carve_stack(Carver& c, long long count, long long rows, long long cols) {
  Quantised m;
  m.ld = (cols + 15) & ~15LL;
  m.q = c.take((size_t)count * rows * m.ld);
  m.s = reinterpret_cast<float*>(c.take((size_t)count * blocks128(rows) * blocks128(cols) * 4));
  return m;
}
SavedExperts carve_saved_experts(uint8_t* base, long long T, long long N, long long K, long long E) {
  Carver c{base};
  SavedExperts v;
  v.offsets = reinterpret_cast<long long*>(c.take((size_t)(E + 1) * 8));
  v.xt = carve(c, K, 128 * group_blocks(T, E), K);
  v.w = carve_stack(c, E, N, K);
  v.bytes = c.off;
  return v;
}
F8Groups groups(const void* offsets, long long E, unsigned flags, bool by_blocks, long long rows) {
  return F8Groups{offsets, (flags & RG_FLAG_OFFSETS64) != 0, E, (flags & RG_FLAG_KEEP_REST) == 0, by_blocks, rows};
}
int grouped(const F8GemmArgs& a, const F8Groups& g, DevPlan* plan, cudaStream_t st) {
  if (!(a.M && a.N)) return a.keep_status ? RG_OK : reset_status(plan, st);
  return launch_f8_grouped(a, g, plan, st, take_fault(), wait_limit_ns()) == cudaSuccess ? RG_OK : RG_ERR_CUDA;
}
// Rows in groups: also the blocks along the columns.
int quantise_groups(QuantArgs a, int type, int form, const void* offsets, long long E, unsigned flags, cudaStream_t st) {
  a.offsets = offsets;
  a.wide = (flags & RG_FLAG_OFFSETS64) != 0;
  a.E = (int)E;
  a.blocks = group_blocks(a.M, E);
  if (!a.K) return RG_OK;
  return launch_quantise_f8(a, type, form, st) == cudaSuccess ? RG_OK : RG_ERR_CUDA;
}
int quantise_stack(QuantArgs a, int type, long long count, cudaStream_t st) {
  a.batch = count;
  return quantise(a, type, RG_F8_TILES, st);
}
F8GemmArgs blocks_args(const Quantised& a, const Quantised& b, void* C, int c_type, long long M, long long N,
                       long long blocks) {
  return F8GemmArgs{a.q, b.q, a.s, b.s, C, a.ld, b.ld, N, blocks, 1, M, N, 128 * blocks, c_type, true, false};
}
QuantArgs quant_args(const void* X, long long ldx, long long M, long long K, const Quantised& rows,
                     const Quantised& columns) {
  return QuantArgs{X, ldx, M, K, rows.q, rows.ld, rows.s, columns.q, columns.ld, columns.s};
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
    const int rc = quantise(QuantArgs{X, ldx, M, K, Q, ldq, S, QT, ldqt, ST}, x_type, form, st);
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
  int rc = quantise(QuantArgs{X, ldx, M, K, x.q, x.ld, x.s, v.xt.q, v.xt.ld, v.xt.s}, x_type,
                    RG_F8_BOTH, st);
  if (!rc)
    rc = quantise(QuantArgs{W, ldw, N, K, v.w.q, v.w.ld, v.w.s, nullptr, 0, nullptr}, w_type,
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
  const Wanted want(flags);
  if ((M && N && (!dY || lddy < N)) || (want.dx && M && K && !dX) || (want.dw && N && K && !dW)) return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const Saved v = carve_saved(static_cast<uint8_t*>(const_cast<void*>(saved)), M, N, K);
  DevPlan* plan = static_cast<DevPlan*>(ws);
  Carver c{static_cast<uint8_t*>(ws) + kCallBlockBytes};
  const Quantised d = carve(c, M, N, M), dt = carve(c, N, M, N);
  if (!want.dx && !want.dw) {
    const int rc = reset_status(plan, st);
    return rc ? rc : finish_call(ws, st, flags);
  }
  int rc = quantise(quant_args(dY, lddy, M, N, d, dt), dy_type, want.form(), st);
  if (!rc && want.dx)  // dX [M][K] = dY [M][N] W [N][K]
    rc = product(gemm_args(d.q, d.ld, d.s, v.w.q, v.w.ld, v.w.s, dX, dy_type, K, M, K, N, false, true), plan, st);
  if (!rc && want.dw) {  // dW [N][K] = dY^T [N][M] (X^T [K][M])^T
    F8GemmArgs a = gemm_args(dt.q, dt.ld, dt.s, v.xt.q, v.xt.ld, v.xt.s, dW, dw_type, K, N, K, M, true, false);
    a.keep_status = want.dx;
    rc = product(a, plan, st);
  }
  return rc ? rc : finish_call(ws, st, flags);
}

int scaled_gemm_act_f8(const uint8_t* A, int64_t lda, const float* SA, const uint8_t* B, int64_t ldb, const float* SB,
                       const void* bias, int bias_type, int act, const void* R, int64_t ldr, void* P, void* C,
                       int c_type, int64_t ldc, int64_t M, int64_t N, int64_t K, unsigned flags, void* ws,
                       size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return RG_ERR_ARG;
  if (!good_type(c_type) || (bias && !good_type(bias_type)) || !good_act(act) || M < 0 || N < 0 || K < 1 ||
      M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return RG_ERR_ARG;
  if (ws_bytes < kCallBlockBytes) return RG_ERR_WORKSPACE;
  if (M && N) {
    if (!C || ldc < N || (R && ldr < N) || !A || !B || !SA || !SB || lda < K || ldb < K || !aligned16(A, lda) ||
        !aligned16(B, ldb) || blocks128(M) * blocks128(N) > INT_MAX / 8)
      return RG_ERR_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const F8Epilogue ep{bias, bias_type, act, R, ldr, P};
  F8GemmArgs a = gemm_args(A, lda, SA, B, ldb, SB, C, c_type, ldc, M, N, K, true, true);
  a.ep = &ep;
  const int rc = product(a, static_cast<DevPlan*>(ws), st);
  return rc ? rc : finish_call(ws, st, flags);
}

size_t linear_act_f8_saved_bytes(int64_t M, int64_t N, int64_t K, int x_type, int act) {
  if (!good_linear(M, N, K) || !K || !good_type(x_type) || !good_act(act)) return 0;
  return carve_saved_act(nullptr, M, N, K, x_type, act).bytes + 256;
}

size_t linear_act_f8_ws_bytes(int64_t M, int64_t N, int64_t K) {
  if (!good_linear(M, N, K) || !K) return 0;
  return linear_f8_ws_bytes(M, N, K) + (((size_t)blocks128(M) * N * 4 + 255) & ~size_t(255));
}

int linear_act_f8(const void* X, int x_type, int64_t ldx, const void* W, int w_type, int64_t ldw, const void* bias,
                  int bias_type, int act, const void* R, int64_t ldr, void* Y, int64_t M, int64_t N, int64_t K,
                  void* saved, size_t saved_bytes, unsigned flags, void* ws, size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || !saved || (reinterpret_cast<uintptr_t>(saved) & 255u) ||
      !good_type(x_type) || !good_type(w_type) || (bias && !good_type(bias_type)) || !good_act(act) ||
      !good_linear(M, N, K) || !K)
    return RG_ERR_ARG;
  if (ws_bytes < linear_act_f8_ws_bytes(M, N, K) || saved_bytes < linear_act_f8_saved_bytes(M, N, K, x_type, act))
    return RG_ERR_WORKSPACE;
  if ((M && (!X || ldx < K)) || (N && (!W || ldw < K)) || (M && N && (!Y || (R && ldr < N)))) return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const SavedAct v = carve_saved_act(static_cast<uint8_t*>(saved), M, N, K, x_type, act);
  const Quantised &xt = v.linear.xt, &w = v.linear.w;
  Carver c{static_cast<uint8_t*>(ws) + kCallBlockBytes};
  const Quantised x = carve(c, M, K, M);
  int rc = quantise(quant_args(X, ldx, M, K, x, xt), x_type, RG_F8_BOTH, st);
  if (!rc) {  // beside X's quantisation
    QuantArgs q = quant_args(W, ldw, N, K, w, Quantised{});
    q.late = M > 0;
    rc = quantise(q, w_type, RG_F8_TILES, st);
  }
  if (!rc) {
    const F8Epilogue ep{bias, bias_type, act, R, ldr, v.p};
    F8GemmArgs a = gemm_args(x.q, x.ld, x.s, w.q, w.ld, w.s, Y, x_type, N, M, N, K, true, true);
    a.ep = &ep;
    rc = product(a, static_cast<DevPlan*>(ws), st);
  }
  return rc ? rc : finish_call(ws, st, flags);
}

int linear_act_f8_backward(const void* dY, int x_type, int64_t lddy, const void* saved, size_t saved_bytes, int act,
                           void* dX, void* dW, int dw_type, void* dbias, int bias_type, int64_t M, int64_t N, int64_t K,
                           unsigned flags, void* ws, size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || !saved || (reinterpret_cast<uintptr_t>(saved) & 255u) ||
      !good_type(x_type) || !good_type(dw_type) || (dbias && !good_type(bias_type)) || !good_act(act) ||
      !good_linear(M, N, K) || !K)
    return RG_ERR_ARG;
  if (ws_bytes < linear_act_f8_ws_bytes(M, N, K) || saved_bytes < linear_act_f8_saved_bytes(M, N, K, x_type, act))
    return RG_ERR_WORKSPACE;
  const Wanted want(flags);
  if ((M && N && (!dY || lddy < N)) || (want.dx && M && !dX) || (want.dw && N && !dW)) return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const SavedAct v = carve_saved_act(static_cast<uint8_t*>(const_cast<void*>(saved)), M, N, K, x_type, act);
  const Quantised &xt = v.linear.xt, &w = v.linear.w;
  DevPlan* plan = static_cast<DevPlan*>(ws);
  Carver c{static_cast<uint8_t*>(ws) + kCallBlockBytes};
  const Quantised d = carve(c, M, N, M), dt = carve(c, N, M, N);
  if (!want.dx && !want.dw && !dbias) {
    const int rc = reset_status(plan, st);
    return rc ? rc : finish_call(ws, st, flags);
  }
  QuantArgs q = quant_args(dY, lddy, M, N, d, dt);
  q.act = act;
  q.P = v.p;
  q.sums = dbias ? reinterpret_cast<float*>(c.take((size_t)blocks128(M) * N * 4)) : nullptr;
  q.out = dbias;
  q.out_type = bias_type;
  // with a slope or sums there is one form
  int rc = quantise(q, x_type, act == RG_ACT_NONE && !dbias ? want.form() : RG_F8_BOTH, st);
  const bool sum = dbias && N && (!M || blocks128(M) > kSumCluster);
  if (!rc && sum &&
      launch_sum_rows(q.sums, M ? blocks128(M) : 0, N, dbias, bias_type, st) != cudaSuccess)
    rc = RG_ERR_CUDA;
  // The sums of rows and the two products read what the quantisation wrote, and
  // nothing of each other's.
  if (!rc && want.dx) {
    F8GemmArgs a = gemm_args(d.q, d.ld, d.s, w.q, w.ld, w.s, dX, x_type, K, M, K, N, false, true);
    a.late = M && N && sum;
    rc = product(a, plan, st);
  }
  if (!rc && want.dw) {
    F8GemmArgs a = gemm_args(dt.q, dt.ld, dt.s, xt.q, xt.ld, xt.s, dW, dw_type, K, N, K, M, true, false);
    a.keep_status = want.dx;
    a.late = M && N && (sum || want.dx);
    rc = product(a, plan, st);
  }
  if (!rc && !want.dx && !want.dw) rc = reset_status(plan, st);
  return rc ? rc : finish_call(ws, st, flags);
}

int quantize_grouped_f8(const void* X, int x_type, int64_t ldx, int64_t M, int64_t K, int form, const void* offsets,
                        int64_t E, uint8_t* Q, int64_t ldq, float* S, uint8_t* QT, int64_t ldqt, float* ST,
                        unsigned flags, void* stream) {
  if (!good_type(x_type) || form < RG_F8_COLUMNS || form > RG_F8_TILES || M < 0 || K < 0 || M > kMaxDim || K > kMaxDim ||
      E < 1 || E > RG_MOE_MAX_EXPERTS)
    return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int rc = RG_OK;
  if (form == RG_F8_TILES) {
    if (M && K && (!X || !Q || !S || ldx < K || ldq < K || blocks128(M) * blocks128(K) > INT_MAX)) return RG_ERR_ARG;
    rc = quantise_stack(QuantArgs{X, ldx, M, K, Q, ldq, S}, x_type, E, st);
  } else {
    const bool both = form == RG_F8_BOTH;
    if (!good_groups(M, E, offsets, flags)) return RG_ERR_ARG;
    if (K && ((M && (!X || ldx < K || (both && (!Q || !S || ldq < K)))) || !QT || !ST ||
              ldqt < 128 * group_blocks(M, E) || (group_blocks(M, E) + 1) * blocks128(K) > INT_MAX))
      return RG_ERR_ARG;
    rc = quantise_groups(QuantArgs{X, ldx, M, K, Q, ldq, S, QT, ldqt, ST}, x_type, form, offsets, E, flags, st);
  }
  if (rc) return rc;
  if ((flags & RG_FLAG_SYNC) && cudaStreamSynchronize(st) != cudaSuccess) return RG_ERR_CUDA;
  return RG_OK;
}

int grouped_gemm_f8(const uint8_t* A, int64_t lda, const float* SA, const uint8_t* B, int64_t ldb, const float* SB,
                    const void* offsets, int64_t E, void* C, int c_type, int64_t ldc, int64_t T, int64_t N, int64_t K,
                    unsigned flags, void* ws, size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return RG_ERR_ARG;
  if (!good_type(c_type) || !good_groups(T, E, offsets, flags) || N < 0 || K < 1 || N > kMaxDim || K > kMaxDim)
    return RG_ERR_ARG;
  if (ws_bytes < kCallBlockBytes) return RG_ERR_WORKSPACE;
  const bool transb = (flags & RG_FLAG_TRANS_B) != 0;
  if (T && N &&
      (!C || ldc < N || !A || !B || !SA || !SB || lda < K || ldb < (transb ? K : N) || !aligned16(A, lda) ||
       !aligned16(B, ldb) || (T / 128 + E + 1) * blocks128(N) > INT_MAX / 8))
    return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const int rc = grouped(gemm_args(A, lda, SA, B, ldb, SB, C, c_type, ldc, T, N, K, transb, true),
                         groups(offsets, E, flags, false, T), static_cast<DevPlan*>(ws), st);
  return rc ? rc : finish_call(ws, st, flags);
}

int grouped_wgrad_f8(const uint8_t* A, int64_t lda, const float* SA, const uint8_t* B, int64_t ldb, const float* SB,
                     const void* offsets, int64_t E, void* C, int c_type, int64_t M, int64_t N, int64_t blocks,
                     unsigned flags, void* ws, size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return RG_ERR_ARG;
  if (!good_type(c_type) || !good_groups(0, E, offsets, flags) || M < 0 || N < 0 || M > kMaxDim || N > kMaxDim ||
      blocks < E || blocks > kMaxDim / 128 || E * M > kMaxDim)
    return RG_ERR_ARG;
  if (ws_bytes < kCallBlockBytes) return RG_ERR_WORKSPACE;
  if (M && N &&
      (!C || !A || !B || !SA || !SB || lda < 128 * blocks || ldb < 128 * blocks || !aligned16(A, lda) ||
       !aligned16(B, ldb) || E * blocks128(M) * blocks128(N) > INT_MAX / 8))
    return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const Quantised a{const_cast<uint8_t*>(A), const_cast<float*>(SA), lda};
  const Quantised b{const_cast<uint8_t*>(B), const_cast<float*>(SB), ldb};
  // the most rows that take so many blocks
  const F8Groups g = groups(offsets, E, flags, true, 128 * (blocks - E) + 127);
  const int rc = grouped(blocks_args(a, b, C, c_type, M, N, blocks), g, static_cast<DevPlan*>(ws), st);
  return rc ? rc : finish_call(ws, st, flags);
}

size_t expert_linear_f8_saved_bytes(int64_t T, int64_t N, int64_t K, int64_t E) {
  return good_expert_linear(T, N, K, E) ? carve_saved_experts(nullptr, T, N, K, E).bytes + 256 : 0;
}

size_t expert_linear_f8_ws_bytes(int64_t T, int64_t N, int64_t K, int64_t E) {
  if (!good_expert_linear(T, N, K, E)) return 0;
  Carver forward{nullptr}, backward{nullptr};
  carve(forward, T, K, T);
  carve(backward, T, N, T);
  carve(backward, N, 128 * group_blocks(T, E), N);
  return kCallBlockBytes + (forward.off > backward.off ? forward.off : backward.off);
}

int expert_linear_f8(const void* X, int x_type, int64_t ldx, const void* W, int w_type, int64_t ldw,
                     const void* offsets, int64_t E, void* Y, int64_t T, int64_t N, int64_t K, void* saved,
                     size_t saved_bytes, unsigned flags, void* ws, size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || !saved || (reinterpret_cast<uintptr_t>(saved) & 255u) ||
      !good_type(x_type) || !good_type(w_type) || !good_expert_linear(T, N, K, E) ||
      !good_groups(T, E, offsets, flags))
    return RG_ERR_ARG;
  if (ws_bytes < expert_linear_f8_ws_bytes(T, N, K, E) || saved_bytes < expert_linear_f8_saved_bytes(T, N, K, E))
    return RG_ERR_WORKSPACE;
  if ((T && (!X || ldx < K)) || (N && (!W || ldw < K)) || (T && N && !Y)) return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const SavedExperts v = carve_saved_experts(static_cast<uint8_t*>(saved), T, N, K, E);
  Carver c{static_cast<uint8_t*>(ws) + kCallBlockBytes};
  const Quantised x = carve(c, T, K, T);
  QuantArgs qx = quant_args(X, ldx, T, K, x, v.xt);
  qx.kept_offsets = v.offsets;
  int rc = quantise_groups(qx, x_type, RG_F8_BOTH, offsets, E, flags, st);
  if (!rc) {  // beside X's quantisation
    QuantArgs q = quant_args(W, ldw, N, K, v.w, Quantised{});
    q.late = true;
    rc = quantise_stack(q, w_type, E, st);
  }
  if (!rc)
    rc = grouped(gemm_args(x.q, x.ld, x.s, v.w.q, v.w.ld, v.w.s, Y, x_type, N, T, N, K, true, true),
                 groups(offsets, E, flags & ~RG_FLAG_KEEP_REST, false, T), static_cast<DevPlan*>(ws), st);
  return rc ? rc : finish_call(ws, st, flags);
}

int expert_linear_f8_backward(const void* dY, int dy_type, int64_t lddy, const void* saved, size_t saved_bytes,
                              const void* offsets, int64_t E, void* dX, void* dW, int dw_type, int64_t T, int64_t N,
                              int64_t K, unsigned flags, void* ws, size_t ws_bytes, void* stream) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || !saved || (reinterpret_cast<uintptr_t>(saved) & 255u) ||
      !good_type(dy_type) || !good_type(dw_type) || !good_expert_linear(T, N, K, E) ||
      !good_groups(T, E, offsets, flags))
    return RG_ERR_ARG;
  if (ws_bytes < expert_linear_f8_ws_bytes(T, N, K, E) || saved_bytes < expert_linear_f8_saved_bytes(T, N, K, E))
    return RG_ERR_WORKSPACE;
  const Wanted want(flags);
  if ((T && N && (!dY || lddy < N)) || (want.dx && T && !dX) || (want.dw && N && !dW)) return RG_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const WorkspaceTurn turn(ws);
  const SavedExperts v = carve_saved_experts(static_cast<uint8_t*>(const_cast<void*>(saved)), T, N, K, E);
  DevPlan* plan = static_cast<DevPlan*>(ws);
  Carver c{static_cast<uint8_t*>(ws) + kCallBlockBytes};
  const Quantised d = carve(c, T, N, T), dt = carve(c, N, 128 * group_blocks(T, E), N);
  if (!want.dx && !want.dw) {
    const int rc = reset_status(plan, st);
    return rc ? rc : finish_call(ws, st, flags);
  }
  const QuantArgs q = quant_args(dY, lddy, T, N, d, dt);
  int rc = want.dw ? quantise_groups(q, dy_type, want.form(), offsets, E, flags, st)
                   : quantise(q, dy_type, RG_F8_ROWS, st);  // blocks along the rows' entries know no groups
  if (!rc && want.dx) {  // dX [T][K] = dY [T][N] W_g [N][K]; nothing to sum without N
    if (N) {
      rc = grouped(gemm_args(d.q, d.ld, d.s, v.w.q, v.w.ld, v.w.s, dX, dy_type, K, T, K, N, false, true),
                   groups(offsets, E, flags & ~RG_FLAG_KEEP_REST, false, T), plan, st);
    } else if (reset_status(plan, st) ||
               (T && cudaMemsetAsync(dX, 0, (size_t)T * K * type_bytes(dy_type), st) != cudaSuccess)) {
      rc = RG_ERR_CUDA;
    }
  }
  if (!rc && want.dw) {  // dW [E][N][K]: per group dY^T X
    F8GemmArgs a = blocks_args(dt, v.xt, dW, dw_type, N, K, group_blocks(T, E));
    a.keep_status = want.dx;
    a.late = want.dx && T && N;  // beside dX, which it does not read
    rc = grouped(a, groups(offsets, E, flags, true, T), plan, st);
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
