"""8-bit products by group: rows sorted by expert, with a weight matrix for each (f8.py has the format and how calls
are made).

offsets [E + 1] (int32 or int64, on the device) says where each group's rows start: group g holds rows offsets[g] to
offsets[g + 1] - 1, from offsets[0] = 0 on.  Groups may be empty, and rows may follow the last one.  Nothing here
reads the offsets on the host: ones that fall, or end past the rows, are a device-side error (ResGemmError, with
sync=False from status()).  The kernel of a product is therefore chosen by all rows of the buffer, and spare ones are
quantised with the others: a buffer not far above what a call holds costs least.

Along the rows, blocks of 128 lie in one group each: group g's start at block offsets[g] // 128 + g, its last one is
filled up with zeros, and a matrix of T rows has T // 128 + E blocks.  quantize_f8 with offsets lays them out.
"""
from __future__ import annotations

import functools

import torch

from . import (RG_ERR_ARG, RG_FLAG_KEEP_REST, RG_FLAG_OFFSETS64, RG_FLAG_SYNC, RG_FLAG_TRANS_B, ResGemmError, _output,
               library)
from .f8 import (_TYPES, _WS_BYTES, F8, _aligned_rows, _backward_flags, _blocks, _check_capture, _device_index, _groups,
                 _launch, _native, _no_grad, _ptr, _rows_of, _scratch, _stack_stride)


def _aligned_stack(q: torch.Tensor):
    """(stack of matrices, row stride) with rows on 16-byte boundaries and no gaps between the matrices, copied only
    where they are not."""
    E, R, C = q.shape
    ld = _stack_stride(q)
    if R == 1 and E == 1:
        ld = (ld + 15) & ~15
    if not ld or ld & 15 or q.data_ptr() & 15:
        ld = (C + 15) & ~15
        c = torch.empty_strided((E, R, C), (R * ld, ld, 1), dtype=F8, device=q.device)
        c.view(torch.uint8).copy_(q.view(torch.uint8))
        return c, ld
    return q, ld


def grouped_gemm_f8(A: torch.Tensor, SA: torch.Tensor, B: torch.Tensor, SB: torch.Tensor, offsets: torch.Tensor,
                    out_dtype: torch.dtype = torch.bfloat16, transb: bool = False, sync: bool = True, out=None,
                    ws: torch.Tensor | None = None) -> torch.Tensor:
    """C [T, N]: every row of A [T, K] times its group's B[g], of B [E, K, N]; with transb, B is given as [E, N, K] and
    the product is with B[g].T.

    A E4M3 with SA [T, ceil(K/128)]; B E4M3 with one scale per 128 x 128 tile of each matrix, SB [E, ceil(K/128),
    ceil(N/128)], transb [E, ceil(N/128), ceil(K/128)]; K at least 1.  Products and sums as in scaled_gemm_f8, one
    rounding to out_dtype.  Rows behind the last group are 0 in a new C; those of a given out stay as they are.  No
    gradient (expert_linear_f8 has one): a backward pass through C raises."""
    where = "grouped_gemm_f8"
    if torch.is_grad_enabled() and (A.requires_grad or SA.requires_grad or B.requires_grad or SB.requires_grad):
        return _no_grad(where, out, lambda: grouped_gemm_f8(A, SA, B, SB, offsets, out_dtype, transb, sync, None, ws),
                        A, SA, B, SB)
    if out is None and ws is None and A.is_cuda:
        C = _native().rows(A, SA, B, SB, offsets, out_dtype, transb, RG_FLAG_SYNC if sync else 0)
        if C is not None:
            return C
    if A.dim() != 2 or B.dim() != 3 or A.dtype != F8 or B.dtype != F8 or not A.shape[1]:
        raise ValueError(f"{where}: A [T, K] and B [E, K, N] (transb: [E, N, K]) float8_e4m3fn expected")
    T, K = A.shape
    E, N, Kb = B.shape if transb else (B.shape[0], B.shape[2], B.shape[1])
    if K != Kb:
        raise ValueError(f"{where}: A and B differ in K")
    t = _TYPES.get(out_dtype)
    if t is None:
        raise ValueError(f"{where}: out_dtype float32, float16 or bfloat16 expected")
    kb, nb = _blocks(K), _blocks(N)
    sb = (E, nb, kb) if transb else (E, kb, nb)
    if SA.dtype != torch.float32 or SB.dtype != torch.float32 or SA.shape != (T, kb) or SB.shape != sb:
        raise ValueError(f"{where}: float32 scales SA {(T, kb)} and SB {sb} expected")
    idx = _device_index(where, A, SA, B, SB, offsets)
    offsets, flags = _groups(where, offsets, E)
    flags |= (RG_FLAG_SYNC if sync else 0) | (RG_FLAG_TRANS_B if transb else 0) | (RG_FLAG_KEEP_REST if out is not None
                                                                                  else 0)
    A, lda = _aligned_rows(A)
    B, ldb = _aligned_stack(B)
    SA, SB = SA.contiguous(), SB.contiguous()
    C = torch.empty((T, N), dtype=out_dtype, device=A.device) if out is None else \
        _output(out, (T, N), out_dtype, A, False, where)
    w = ws if ws is not None else _scratch(_WS_BYTES, idx)
    _launch(idx, where, library().grouped_gemm_f8, A.data_ptr(), lda, SA.data_ptr(), B.data_ptr(), ldb, SB.data_ptr(),
            offsets.data_ptr(), E, C.data_ptr(), t, N, T, N, K, flags, w.data_ptr(), w.numel())
    return C


def grouped_wgrad_f8(A: torch.Tensor, SA: torch.Tensor, B: torch.Tensor, SB: torch.Tensor, offsets: torch.Tensor,
                     out_dtype: torch.dtype = torch.float32, sync: bool = True, out=None,
                     ws: torch.Tensor | None = None) -> torch.Tensor:
    """C [E, M, N]: per group the sum over its rows t of A[:, t] B[:, t]^T, for operands stored along the rows, in blocks
    of one group each: A [M, 128 NB] E4M3 with SA [M, NB], B [N, 128 NB] with SB [N, NB], as quantize_f8(X, "columns",
    offsets=offsets) gives them (NB = T // 128 + E).  0 for a group without rows.  No gradient."""
    where = "grouped_wgrad_f8"
    if torch.is_grad_enabled() and (A.requires_grad or SA.requires_grad or B.requires_grad or SB.requires_grad):
        return _no_grad(where, out, lambda: grouped_wgrad_f8(A, SA, B, SB, offsets, out_dtype, sync, None, ws),
                        A, SA, B, SB)
    if out is None and ws is None and A.is_cuda:
        C = _native().sums(A, SA, B, SB, offsets, out_dtype, RG_FLAG_SYNC if sync else 0)
        if C is not None:
            return C
    if A.dim() != 2 or B.dim() != 2 or A.dtype != F8 or B.dtype != F8 or A.shape[1] != B.shape[1] or \
            A.shape[1] % 128:
        raise ValueError(f"{where}: A [M, 128 NB] and B [N, 128 NB] float8_e4m3fn expected")
    t = _TYPES.get(out_dtype)
    if t is None:
        raise ValueError(f"{where}: out_dtype float32, float16 or bfloat16 expected")
    M, N, nb = A.shape[0], B.shape[0], A.shape[1] // 128
    if SA.dtype != torch.float32 or SB.dtype != torch.float32 or SA.shape != (M, nb) or SB.shape != (N, nb):
        raise ValueError(f"{where}: float32 scales SA {(M, nb)} and SB {(N, nb)} expected")
    E = offsets.shape[0] - 1 if offsets.dim() == 1 else 0
    idx = _device_index(where, A, SA, B, SB, offsets)
    offsets, flags = _groups(where, offsets, E)
    if nb < E:
        raise ValueError(f"{where}: at least a block for each group expected")
    A, lda = _aligned_rows(A)
    B, ldb = _aligned_rows(B)
    SA, SB = SA.contiguous(), SB.contiguous()
    C = torch.empty((E, M, N), dtype=out_dtype, device=A.device) if out is None else \
        _output(out, (E, M, N), out_dtype, A, False, where)
    w = ws if ws is not None else _scratch(_WS_BYTES, idx)
    _launch(idx, where, library().grouped_wgrad_f8, A.data_ptr(), lda, SA.data_ptr(), B.data_ptr(), ldb, SB.data_ptr(),
            offsets.data_ptr(), E, C.data_ptr(), t, M, N, nb, flags | (RG_FLAG_SYNC if sync else 0), w.data_ptr(),
            w.numel())
    return C


@functools.lru_cache(maxsize=512)
def _expert_bytes(T, N, K, E):
    """(bytes kept between the passes, workspace bytes)."""
    lib = library()
    saved, need = int(lib.expert_linear_f8_saved_bytes(T, N, K, E)), int(lib.expert_linear_f8_ws_bytes(T, N, K, E))
    if not saved or not need:
        raise ResGemmError(RG_ERR_ARG, "expert_linear_f8")
    return saved, need


class _ExpertGrad(torch.autograd.Function):
    """expert_linear_f8 with expert_linear_f8_backward as its gradient; `saved` receives what the latter reads."""

    @staticmethod
    def forward(ctx, X, W, offsets, sync, ws, saved):
        Y, (kept, *ctx.rest) = expert_linear_f8(X, W, offsets, sync, ws)
        ctx.save_for_backward(kept, offsets)  # offsets: so that autograd notices where they change
        ctx.call = sync, W.dtype, ws
        saved.extend((kept, *ctx.rest))
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        _check_capture("expert_linear_f8", ctx)
        return (*expert_linear_f8_backward(dY, (ctx.saved_tensors[0], *ctx.rest), *ctx.call, *ctx.needs_input_grad[:2]),
                None, None, None, None)


def expert_linear_f8(X: torch.Tensor, W: torch.Tensor, offsets: torch.Tensor, sync: bool = True,
                     ws: torch.Tensor | None = None):
    """(Y, saved): linear_f8 by group: Y [T, N] = X W[g]^T for each group's rows of X [T, K], weights W [E, N, K], in X's
    dtype (both float32, float16 or bfloat16); rows behind the last group are 0.  `saved` is what
    expert_linear_f8_backward needs, a copy of the offsets among it: the caller's own may be rewritten for another call
    in between (not under autograd, whose backward pass refuses tensors that have changed).  Where X or W requires a
    gradient autograd calls expert_linear_f8_backward for Y, with W's gradient in W's dtype."""
    if torch.is_grad_enabled() and (X.requires_grad or W.requires_grad):
        saved = []
        return _ExpertGrad.apply(X, W, offsets, sync, ws, saved), tuple(saved)
    if X.is_cuda and ws is None:
        r = _native().expert(X, W, offsets, RG_FLAG_SYNC if sync else 0)
        if r is not None:
            return r
    where = "expert_linear_f8"
    tx, tw = _TYPES.get(X.dtype), _TYPES.get(W.dtype)
    if tx is None or tw is None or X.dim() != 2 or W.dim() != 3 or X.shape[1] != W.shape[2] or not X.shape[1]:
        raise ValueError(f"{where}: X [T, K] and W [E, N, K] float32, float16 or bfloat16 expected")
    idx = _device_index(where, X, W, offsets)
    (T, K), (E, N, _) = X.shape, W.shape
    offsets, flags = _groups(where, offsets, E)
    nsaved, need = _expert_bytes(T, N, K, E)
    X, ldx = _rows_of(X)
    ldw = _stack_stride(W)
    if not ldw:
        W, ldw = W.contiguous(), K
    Y = torch.empty((T, N), dtype=X.dtype, device=X.device)
    kept = torch.empty(nsaved, dtype=torch.uint8, device=X.device)
    w = ws if ws is not None else _scratch(need, idx)
    _launch(idx, where, library().expert_linear_f8, X.data_ptr(), tx, ldx, W.data_ptr(), tw, ldw, offsets.data_ptr(), E,
            Y.data_ptr(), T, N, K, kept.data_ptr(), nsaved, flags | (RG_FLAG_SYNC if sync else 0), w.data_ptr(),
            w.numel())
    return Y, (kept, None, T, N, K, E)  # None: the copy of the offsets with which the buffer begins


def expert_linear_f8_backward(dY: torch.Tensor, saved, sync: bool = True, dw_dtype: torch.dtype = torch.float32,
                              ws: torch.Tensor | None = None, dx: bool = True, dw: bool = True):
    """(dX, dW) of expert_linear_f8 for the output's gradient dY [T, N]: dX = dY W[g] with dY quantised along N, in dY's
    dtype, 0 behind the last group, and dW [E, N, K] = dY^T X over each group's rows, both quantised along them, in
    dw_dtype.  With dx or dw false that gradient is not computed, and None."""
    kept, offsets, T, N, K, E = saved
    flags = _backward_flags(sync, dx, dw)
    if dY.is_cuda and ws is None:
        r = _native().expert_backward(dY, kept, offsets, T, N, K, E, dw_dtype, flags)
        if r is not None:
            return r
    where = "expert_linear_f8_backward"
    t, tw = _TYPES.get(dY.dtype), _TYPES.get(dw_dtype)
    if t is None or tw is None or dY.shape != (T, N):
        raise ValueError(f"{where}: dY with the output's shape, float32, float16 or bfloat16, expected")
    if offsets is None:
        idx, offsets, wide = _device_index(where, dY, kept), kept, RG_FLAG_OFFSETS64
    else:
        idx, (offsets, wide) = _device_index(where, dY, kept, offsets), _groups(where, offsets, E)
    need = _expert_bytes(T, N, K, E)[1]
    dY, lddy = _rows_of(dY)
    dX = torch.empty((T, K), dtype=dY.dtype, device=dY.device) if dx else None
    dW = torch.empty((E, N, K), dtype=dw_dtype, device=dY.device) if dw else None
    w = ws if ws is not None else _scratch(need, idx)
    _launch(idx, where, library().expert_linear_f8_backward, dY.data_ptr(), t, lddy, kept.data_ptr(), kept.numel(),
            offsets.data_ptr(), E, _ptr(dX), _ptr(dW), tw, T, N, K, flags | wide, w.data_ptr(), w.numel())
    return dX, dW
