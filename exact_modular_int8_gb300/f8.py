"""8-bit block-scaled operators: quantisation, matrix product, linear layer, mixture-of-experts layer.

The format: E4M3 values (``torch.float8_e4m3fn``) with one float32 scale for every 128 values along the
contraction, or for every 128 x 128 tile of a weight matrix; an entry stands for value * scale.  Argument
marshalling only, as in the rest of the binding: every step runs in the library's kernels on the current
stream.  Quantised matrices have rows that start on 16-byte boundaries, which is what the product
reads; operands from elsewhere that do not are copied into such rows first.

With sync=False a call only enqueues its work, and errors found on the device are read with status() before
the next call on that stream.  Calls can be captured into CUDA graphs (with sync=False): their scratch then
belongs to the graph, and a status can be read from a workspace passed as ws (a uint8 tensor; its size is what
the library's *_ws_bytes functions give, 4096 for scaled_gemm_f8).
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os

import torch

from . import (LIB_PATH, RG_ERR_ARG, RG_ERR_RANGE, RG_F8_BOTH, RG_F8_COLUMNS, RG_F8_ROWS, RG_F8_TILES, RG_FLAG_SYNC,
               RG_FLAG_TILE_B, RG_FLAG_TRANS_B, RG_TYPE_BF16, RG_TYPE_F16, RG_TYPE_F32, ResGemmError, _check, _output,
               _ws_cache, capturing, library, workspace)

BLOCK = 128
F8 = torch.float8_e4m3fn
_TYPES = {torch.float32: RG_TYPE_F32, torch.float16: RG_TYPE_F16, torch.bfloat16: RG_TYPE_BF16}
_FORMS = {"rows": RG_F8_ROWS, "columns": RG_F8_COLUMNS, "both": RG_F8_BOTH, "tiles": RG_F8_TILES}
_WS_BYTES = 4096


def _native():
    """The native call path (csrc/python/f8_call.c), set up once."""
    global _call
    if _call is None:
        lib = library()
        path = os.path.join(os.path.dirname(LIB_PATH), "f8_call.so")
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with `python -m exact_modular_int8_gb300.build`")
        loader = importlib.machinery.ExtensionFileLoader("f8_call", path)
        m = importlib.util.module_from_spec(importlib.util.spec_from_file_location("f8_call", path, loader=loader))
        loader.exec_module(m)
        address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
        entries = (lib.quantize_f8, lib.scaled_gemm_f8, lib.linear_f8, lib.linear_f8_backward,
                   lib.linear_f8_saved_bytes, lib.linear_f8_ws_bytes, lib.rg_stream_capturing)
        m.setup(tuple(address(f) for f in entries), (torch.float32, torch.float16, torch.bfloat16), F8, torch.uint8,
                torch.empty, torch.empty_strided, torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice, _ws_cache,
                _check)
        _call = m
    return _call


_call = None


class _LinearGrad(torch.autograd.Function):
    """linear_f8 with linear_f8_backward as its gradient; `saved` receives what the latter reads."""

    @staticmethod
    def forward(ctx, X, W, sync, ws, saved):
        Y, (kept, *ctx.sizes) = linear_f8(X, W, sync, ws)
        ctx.save_for_backward(kept)
        ctx.call = sync, W.dtype, ws
        saved.extend((kept, *ctx.sizes))
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        return (*linear_f8_backward(dY, (*ctx.saved_tensors, *ctx.sizes), *ctx.call), None, None, None)


class _NoGrad(torch.autograd.Function):
    """A call without a gradient, on tensors that require one: a backward pass through its result raises, where
    a plain result would cut the gradient unnoticed."""

    @staticmethod
    def forward(ctx, where, call, *tensors):
        ctx.where = where
        return call()

    @staticmethod
    def backward(ctx, _):
        raise NotImplementedError(f"{ctx.where} has no gradient; linear_f8 has one")


def _no_grad(where: str, out, call, *tensors):
    if out is not None:
        raise ValueError(f"{where}: out takes no part in differentiation: call under torch.no_grad()")
    return _NoGrad.apply(where, call, *tensors)


def _blocks(x: int) -> int:
    return (x + BLOCK - 1) // BLOCK


def _device_index(where: str, *ts) -> int:
    """The index of the CUDA device that holds all of the tensors."""
    idx = ts[0].get_device()
    for t in ts:
        if t.get_device() != idx or idx < 0:
            raise ValueError(f"{where}: tensors on one CUDA device expected")
    return idx


def _launch(idx: int, where: str, f, *args):
    """The library call f(*args, current stream of device idx) with that device current.  (The raw handle and
    the plain device check take 0.2 us; torch.cuda's Stream object and device context take ten times that.)"""
    stream = torch._C._cuda_getCurrentRawStream(idx)
    if torch._C._cuda_getDevice() == idx:
        rc = f(*args, stream)
    else:
        with torch.cuda.device(idx):
            rc = f(*args, stream)
    if rc:
        _check(rc, where)


def _scratch(nbytes: int, idx: int) -> torch.Tensor:
    """The cached workspace of the device's current stream, or the graph's own (see workspace())."""
    w = None if capturing(idx) else _ws_cache.get((idx, torch._C._cuda_getCurrentRawStream(idx)))
    return w if w is not None and w.numel() >= nbytes else workspace(nbytes, torch.device("cuda", idx))


def _empty_rows(m: int, k: int, device) -> torch.Tensor:
    """[m, k] E4M3 with rows on 16-byte boundaries."""
    return torch.empty_strided((m, k), ((k + 15) & ~15, 1), dtype=F8, device=device)


def _row_stride(t: torch.Tensor) -> int:
    """The row stride of a matrix whose rows are contiguous, else 0 (a stride is immaterial with one row)."""
    (m, k), (s0, s1) = t.shape, t.stride()
    if s1 != 1 and k > 1:
        return 0
    if m <= 1:
        return k or 1
    return s0 if s0 >= k else 0


def _aligned_rows(q: torch.Tensor):
    """(matrix, row stride) with rows on 16-byte boundaries, copied only where they are not."""
    ld = _row_stride(q)
    if q.shape[0] <= 1:
        ld = (ld + 15) & ~15
    if not ld or ld & 15 or q.data_ptr() & 15:
        c = _empty_rows(q.shape[0], q.shape[1], q.device)
        c.view(torch.uint8).copy_(q.view(torch.uint8))
        return c, (q.shape[1] + 15) & ~15
    return q, ld


def quantize_f8(X: torch.Tensor, form: str = "rows", sync: bool = True):
    """E4M3 values and float32 scales of a float32, float16 or bfloat16 matrix X [M, K].

    form "rows":    Q [M, K], S [M, ceil(K/128)]: blocks of 128 along each row
         "columns": Q [K, M], S [K, ceil(M/128)]: the same of X.T
         "both":    (Q, S, Qt, St), the two of them from one read of X
         "tiles":   Q [M, K], S [ceil(M/128), ceil(K/128)]: 128 x 128 tiles
    Per block, a = max |x| (at least 2^-60), S = a / 448, Q = 448 x / a to the nearest E4M3 value, ties to
    even; an inf or NaN makes its whole block NaN.  To autograd the results are constants."""
    f = _FORMS.get(form)
    if f is None:
        raise ValueError(f"quantize_f8: form must be one of {', '.join(_FORMS)}")
    if X.is_cuda:
        r = _native().quantize(X, f, RG_FLAG_SYNC if sync else 0)
        if r is not None:
            return r
    t = _TYPES.get(X.dtype)
    if t is None or X.dim() != 2:
        raise ValueError("quantize_f8: X [M, K] float32, float16 or bfloat16 expected")
    idx = _device_index("quantize_f8", X)
    M, K = X.shape
    ldx = _row_stride(X)
    if not ldx:
        X = X.contiguous()
        ldx = K
    dev = X.device
    q = s = qt = st = qp = sp = qtp = stp = None
    if f != RG_F8_COLUMNS:
        q = _empty_rows(M, K, dev)
        s = torch.empty((_blocks(M) if f == RG_F8_TILES else M, _blocks(K)), dtype=torch.float32, device=dev)
        qp, sp = q.data_ptr(), s.data_ptr()
    if f == RG_F8_COLUMNS or f == RG_F8_BOTH:
        qt = _empty_rows(K, M, dev)
        st = torch.empty((K, _blocks(M)), dtype=torch.float32, device=dev)
        qtp, stp = qt.data_ptr(), st.data_ptr()
    _launch(idx, "quantize_f8", library().quantize_f8, X.data_ptr(), t, ldx, M, K, f, qp, (K + 15) & ~15, sp, qtp,
            (M + 15) & ~15, stp, RG_FLAG_SYNC if sync else 0)
    if f == RG_F8_BOTH:
        return q, s, qt, st
    return (qt, st) if f == RG_F8_COLUMNS else (q, s)


def scaled_gemm_f8(A: torch.Tensor, SA: torch.Tensor, B: torch.Tensor, SB: torch.Tensor,
                   out_dtype: torch.dtype = torch.bfloat16, transb: bool = False, sync: bool = True, out=None,
                   ws: torch.Tensor | None = None) -> torch.Tensor:
    """C = A @ B for block-scaled operands; with transb, B is given as [N, K] and C = A @ B.T.

    A [M, K] E4M3 with SA [M, ceil(K/128)].  B's scales are per 128 x 128 tile of B or per 128 values along
    the contraction, told apart by shape: transb SB [ceil(N/128), ceil(K/128)] or [N, ceil(K/128)], else
    [ceil(K/128), ceil(N/128)] or [ceil(K/128), N] (N = 1 is either).  Products per block on the tensor
    cores, scales and sums in float32, one rounding to out_dtype (float32, float16 or bfloat16).  No gradient: a
    backward pass through C raises."""
    if torch.is_grad_enabled() and (A.requires_grad or SA.requires_grad or B.requires_grad or SB.requires_grad):
        return _no_grad("scaled_gemm_f8", out,
                        lambda: scaled_gemm_f8(A, SA, B, SB, out_dtype, transb, sync, None, ws), A, SA, B, SB)
    if out is None and ws is None and A.is_cuda:
        C = _native().gemm(A, SA, B, SB, out_dtype, transb, RG_FLAG_SYNC if sync else 0)
        if C is not None:
            return C
    if A.dim() != 2 or B.dim() != 2 or A.dtype != F8 or B.dtype != F8:
        raise ValueError("scaled_gemm_f8: A [M, K] and B [K, N] (transb: [N, K]) float8_e4m3fn expected")
    M, K = A.shape
    N, Kb = B.shape if transb else (B.shape[1], B.shape[0])
    if K != Kb:
        raise ValueError("scaled_gemm_f8: A and B differ in K")
    t = _TYPES.get(out_dtype)
    if t is None:
        raise ValueError("scaled_gemm_f8: out_dtype float32, float16 or bfloat16 expected")
    kb, nb = _blocks(K), _blocks(N)
    tile, row = ((nb, kb), (N, kb)) if transb else ((kb, nb), (kb, N))
    is_tile = SB.shape == tile
    if SA.dtype != torch.float32 or SB.dtype != torch.float32 or SA.shape != (M, kb) or \
            not (is_tile or SB.shape == row):
        raise ValueError(f"scaled_gemm_f8: float32 scales SA {(M, kb)} and SB {tile} or {row} expected")
    idx = _device_index("scaled_gemm_f8", A, SA, B, SB)
    flags = (RG_FLAG_SYNC if sync else 0) | (RG_FLAG_TRANS_B if transb else 0) | (RG_FLAG_TILE_B if is_tile else 0)
    A, lda = _aligned_rows(A)
    B, ldb = _aligned_rows(B)
    SA, SB = SA.contiguous(), SB.contiguous()
    C = torch.empty((M, N), dtype=out_dtype, device=A.device) if out is None else \
        _output(out, (M, N), out_dtype, A, False, "scaled_gemm_f8")
    w = ws if ws is not None else _scratch(_WS_BYTES, idx)
    _launch(idx, "scaled_gemm_f8", library().scaled_gemm_f8, A.data_ptr(), lda, SA.data_ptr(), B.data_ptr(), ldb,
            SB.data_ptr(), C.data_ptr(), t, N, M, N, K, flags, w.data_ptr(), w.numel())
    return C


@functools.lru_cache(maxsize=512)
def _linear_bytes(M, N, K):
    """(bytes kept between the passes, workspace bytes)."""
    lib = library()
    saved, need = int(lib.linear_f8_saved_bytes(M, N, K)), int(lib.linear_f8_ws_bytes(M, N, K))
    if not saved or not need:
        raise ResGemmError(RG_ERR_ARG, "linear_f8")
    return saved, need


def _rows_of(t: torch.Tensor):
    """(matrix with contiguous rows, row stride), copied only where its rows are not."""
    ld = _row_stride(t)
    return (t, ld) if ld else (t.contiguous(), t.shape[1])


def linear_f8(X: torch.Tensor, W: torch.Tensor, sync: bool = True, ws: torch.Tensor | None = None):
    """(Y, saved): Y = X W^T with X [M, K] quantised along K and the weights W [N, K] in 128 x 128 tiles, in X's
    dtype (both float32, float16 or bfloat16).  `saved` is what linear_f8_backward needs: one buffer with X
    quantised along M and the quantised weights.  One library call; the same as quantize_f8(X, "both"),
    quantize_f8(W, "tiles") and scaled_gemm_f8.  Where X or W requires a gradient autograd calls
    linear_f8_backward for Y, with W's gradient in W's dtype."""
    if torch.is_grad_enabled() and (X.requires_grad or W.requires_grad):
        saved = []
        return _LinearGrad.apply(X, W, sync, ws, saved), tuple(saved)
    if X.is_cuda and ws is None:
        r = _native().linear(X, W, RG_FLAG_SYNC if sync else 0)
        if r is not None:
            return r
    tx, tw = _TYPES.get(X.dtype), _TYPES.get(W.dtype)
    if tx is None or tw is None or X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[1]:
        raise ValueError("linear_f8: X [M, K] and W [N, K] float32, float16 or bfloat16 expected")
    idx = _device_index("linear_f8", X, W)
    (M, K), N = X.shape, W.shape[0]
    nsaved, need = _linear_bytes(M, N, K)
    X, ldx = _rows_of(X)
    W, ldw = _rows_of(W)
    dev = X.device
    Y = torch.empty((M, N), dtype=X.dtype, device=dev)
    kept = torch.empty(nsaved, dtype=torch.uint8, device=dev)
    w = ws if ws is not None else _scratch(need, idx)
    _launch(idx, "linear_f8", library().linear_f8, X.data_ptr(), tx, ldx, W.data_ptr(), tw, ldw, Y.data_ptr(), M, N, K,
            kept.data_ptr(), nsaved, RG_FLAG_SYNC if sync else 0, w.data_ptr(), w.numel())
    return Y, (kept, M, N, K)


def linear_f8_backward(dY: torch.Tensor, saved, sync: bool = True, dw_dtype: torch.dtype = torch.float32,
                       ws: torch.Tensor | None = None):
    """(dX, dW) of linear_f8 for the output's gradient dY [M, N]: dX = dY W with dY quantised along N, in dY's
    dtype, and dW = dY^T X with both quantised along M, in dw_dtype."""
    kept, M, N, K = saved
    if dY.is_cuda and ws is None:
        r = _native().backward(dY, kept, M, N, K, dw_dtype, RG_FLAG_SYNC if sync else 0)
        if r is not None:
            return r
    t, tw = _TYPES.get(dY.dtype), _TYPES.get(dw_dtype)
    if t is None or tw is None or dY.shape != (M, N):
        raise ValueError("linear_f8_backward: dY with the output's shape, float32, float16 or bfloat16, expected")
    idx = _device_index("linear_f8_backward", dY, kept)
    need = _linear_bytes(M, N, K)[1]
    dY, lddy = _rows_of(dY)
    dX = torch.empty((M, K), dtype=dY.dtype, device=dY.device)
    dW = torch.empty((N, K), dtype=dw_dtype, device=dY.device)
    w = ws if ws is not None else _scratch(need, idx)
    _launch(idx, "linear_f8_backward", library().linear_f8_backward, dY.data_ptr(), t, lddy, kept.data_ptr(),
            kept.numel(), dX.data_ptr(), dW.data_ptr(), tw, M, N, K, RG_FLAG_SYNC if sync else 0, w.data_ptr(),
            w.numel())
    return dX, dW


MOE_MAX_TOKENS = 64


@functools.lru_cache(maxsize=512)
def _moe_ws_bytes(T, H, I, E, top_k) -> int:  # noqa: E741
    return int(library().moe_layer_f8_ws_bytes(T, H, I, E, top_k))


def moe_layer_f8(X: torch.Tensor, WR: torch.Tensor, W13: torch.Tensor, S13: torch.Tensor, W2: torch.Tensor,
                 S2: torch.Tensor, top_k: int, renorm: bool = True, sync: bool = True, out=None,
                 ws: torch.Tensor | None = None) -> torch.Tensor:
    """Y [T, H]: a mixture-of-experts layer with 8-bit expert weights for at most 64 tokens X [T, H] (float16 or
    bfloat16): softmax router WR [E, H] (X's dtype), the top_k experts of each token (ties: the lower index),
    their SwiGLU outputs summed with the router's probabilities, divided by the taken ones' sum if renorm.

    W13 [E, 2I, H] E4M3 holds each expert's gate rows, then its up rows, with S13 [E, ceil(2I/128),
    ceil(H/128)]; W2 [E, H, I] with S2 [E, ceil(H/128), ceil(I/128)]: per expert what quantize_f8(W, "tiles")
    gives.  H and I are multiples of 16.  No gradient: a backward pass through Y raises."""
    if torch.is_grad_enabled() and any(t.requires_grad for t in (X, WR, W13, S13, W2, S2)):
        return _no_grad("moe_layer_f8", out,
                        lambda: moe_layer_f8(X, WR, W13, S13, W2, S2, top_k, renorm, sync, None, ws),
                        X, WR, W13, S13, W2, S2)
    if X.dim() != 2 or X.dtype not in (torch.float16, torch.bfloat16) or WR.dtype != X.dtype:
        raise ValueError("moe_layer_f8: X [T, H] and WR [E, H] of one dtype, float16 or bfloat16, expected")
    if W13.dtype != F8 or W2.dtype != F8 or S13.dtype != torch.float32 or S2.dtype != torch.float32:
        raise ValueError("moe_layer_f8: float8_e4m3fn weights with float32 scales expected")
    T, H = X.shape
    if W2.dim() != 3 or W2.shape[1] != H:
        raise ValueError("moe_layer_f8: W2 [E, H, I] expected")
    E, I = W2.shape[0], W2.shape[2]  # noqa: E741
    if WR.shape != (E, H) or W13.shape != (E, 2 * I, H):
        raise ValueError("moe_layer_f8: WR [E, H] and W13 [E, 2I, H] expected")
    if S13.shape != (E, _blocks(2 * I), _blocks(H)) or S2.shape != (E, _blocks(H), _blocks(I)):
        raise ValueError("moe_layer_f8: one scale per 128 x 128 tile expected")
    idx = _device_index("moe_layer_f8", X, WR, W13, S13, W2, S2)
    X, WR, W13, S13, W2, S2 = (_start16(t) for t in (X, WR, W13, S13, W2, S2))
    Y = torch.empty((T, H), dtype=X.dtype, device=X.device) if out is None else \
        _output(out, (T, H), X.dtype, X, False, "moe_layer_f8")
    need = _moe_ws_bytes(T, H, I, E, int(top_k))
    if not need:
        raise ResGemmError(RG_ERR_RANGE if T > MOE_MAX_TOKENS else RG_ERR_ARG, "moe_layer_f8")
    w = ws if ws is not None else _scratch(need, idx)
    _launch(idx, "moe_layer_f8", library().moe_layer_f8, X.data_ptr(), _TYPES[X.dtype], WR.data_ptr(), W13.data_ptr(),
            S13.data_ptr(), W2.data_ptr(), S2.data_ptr(), Y.data_ptr(), T, H, I, E, int(top_k), int(renorm),
            RG_FLAG_SYNC if sync else 0, w.data_ptr(), w.numel())
    return Y


def _start16(t: torch.Tensor) -> torch.Tensor:
    """Contiguous, starting on a 16-byte boundary."""
    t = t.contiguous()
    return t if t.data_ptr() & 15 == 0 else t.clone()
