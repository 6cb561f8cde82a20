"""8-bit products with an epilogue: bias, activation and residual (f8.py has the format and how calls are made).

The activations, on p = X W^T + bias in float32:
    None         p
    "relu"       p where p > 0, else 0
    "silu"       p / (1 + exp(-p))
    "gelu"       p (1 + erf(p / sqrt 2)) / 2
    "gelu_tanh"  p (1 + tanh(sqrt(2 / pi) (p + 0.044715 p^3))) / 2
"""
from __future__ import annotations

import functools

import torch

from . import (RG_ACT_GELU, RG_ACT_GELU_TANH, RG_ACT_NONE, RG_ACT_RELU, RG_ACT_SILU, RG_ERR_ARG, RG_FLAG_SYNC,
               ResGemmError, _output, library)
from .f8 import (_TYPES, _WS_BYTES, F8, _aligned_rows, _backward_flags, _blocks, _check_capture, _device_index, _launch,
                 _native, _no_grad, _ptr, _rows_of, _scratch)

_grad_enabled = torch.is_grad_enabled
_ACTS = {None: RG_ACT_NONE, "relu": RG_ACT_RELU, "silu": RG_ACT_SILU, "gelu": RG_ACT_GELU,
         "gelu_tanh": RG_ACT_GELU_TANH}


def _act(where: str, act) -> int:
    a = _ACTS.get(act)
    if a is None:
        raise ValueError(f"{where}: act must be None or one of {', '.join(k for k in _ACTS if k)}")
    return a


def _beside(where: str, M: int, N: int, bias, residual, dtype):
    """(bias contiguous or None, its type, residual with contiguous rows or None, its row stride)"""
    tb = 0
    if bias is not None:
        tb = _TYPES.get(bias.dtype)
        if tb is None or bias.shape != (N,):
            raise ValueError(f"{where}: bias [N] float32, float16 or bfloat16 expected")
        bias = bias.contiguous()
    ldr = 0
    if residual is not None:
        if residual.dtype != dtype or residual.shape != (M, N):
            raise ValueError(f"{where}: residual {(M, N)} of the output's dtype expected")
        residual, ldr = _rows_of(residual)
    return bias, tb, residual, ldr


def _there(*ts):
    return [t for t in ts if t is not None]


def _differentiable(A, B, C, D, bias, residual) -> bool:
    return _grad_enabled() and (
        A.requires_grad or B.requires_grad or C.requires_grad or D.requires_grad
        or (bias is not None and bias.requires_grad) or (residual is not None and residual.requires_grad))


def scaled_gemm_act_f8(A: torch.Tensor, SA: torch.Tensor, B: torch.Tensor, SB: torch.Tensor,
                       bias: torch.Tensor | None = None, act: str | None = None,
                       residual: torch.Tensor | None = None, pre: bool = False,
                       out_dtype: torch.dtype = torch.bfloat16, sync: bool = True, out=None,
                       ws: torch.Tensor | None = None):
    """C = act(A @ B.T + bias) + residual for block-scaled operands; with pre, (C, P), P = A @ B.T + bias.

    A [M, K] E4M3 with SA [M, ceil(K/128)]; weights B [N, K] with SB [ceil(N/128), ceil(K/128)], one scale per 128
    x 128 tile; K at least 1.  bias [N] in float32, float16 or bfloat16; residual [M, N] in out_dtype, which C and P
    are rounded to once.  out may be the residual itself, which it then replaces.  No gradient (linear_act_f8 has
    one): a backward pass through C raises."""
    if _differentiable(A, SA, B, SB, bias, residual):
        return _no_grad("scaled_gemm_act_f8", out,
                        lambda: scaled_gemm_act_f8(A, SA, B, SB, bias, act, residual, pre, out_dtype, sync, None, ws),
                        *_there(A, SA, B, SB, bias, residual))
    where = "scaled_gemm_act_f8"
    a = _act(where, act)
    if out is None and ws is None and A.is_cuda:
        r = _native().act(A, SA, B, SB, bias, a, residual, pre, out_dtype, RG_FLAG_SYNC if sync else 0)
        if r is not None:
            return r
    if A.dim() != 2 or B.dim() != 2 or A.dtype != F8 or B.dtype != F8 or A.shape[1] != B.shape[1] or not A.shape[1]:
        raise ValueError(f"{where}: A [M, K] and B [N, K] float8_e4m3fn expected")
    (M, K), N = A.shape, B.shape[0]
    t = _TYPES.get(out_dtype)
    if t is None:
        raise ValueError(f"{where}: out_dtype float32, float16 or bfloat16 expected")
    if SA.dtype != torch.float32 or SB.dtype != torch.float32 or SA.shape != (M, _blocks(K)) or \
            SB.shape != (_blocks(N), _blocks(K)):
        raise ValueError(f"{where}: float32 scales SA {(M, _blocks(K))} and SB {(_blocks(N), _blocks(K))} expected")
    idx = _device_index(where, A, SA, B, SB, *_there(bias, residual))
    bias, tb, residual, ldr = _beside(where, M, N, bias, residual, out_dtype)
    A, lda = _aligned_rows(A)
    B, ldb = _aligned_rows(B)
    SA, SB = SA.contiguous(), SB.contiguous()
    C = torch.empty((M, N), dtype=out_dtype, device=A.device) if out is None else \
        _output(out, (M, N), out_dtype, A, False, where)
    P = torch.empty((M, N), dtype=out_dtype, device=A.device) if pre else None
    w = ws if ws is not None else _scratch(_WS_BYTES, idx)
    _launch(idx, where, library().scaled_gemm_act_f8, A.data_ptr(), lda, SA.data_ptr(), B.data_ptr(), ldb,
            SB.data_ptr(), _ptr(bias), tb, a, _ptr(residual), ldr, _ptr(P), C.data_ptr(), t, N, M, N, K,
            RG_FLAG_SYNC if sync else 0, w.data_ptr(), w.numel())
    return (C, P) if pre else C


@functools.lru_cache(maxsize=512)
def _linear_act_bytes(M, N, K, t, act):
    """(bytes kept between the passes, workspace bytes)."""
    lib = library()
    saved, need = int(lib.linear_act_f8_saved_bytes(M, N, K, t, act)), int(lib.linear_act_f8_ws_bytes(M, N, K))
    if not saved or not need:
        raise ResGemmError(RG_ERR_ARG, "linear_act_f8")
    return saved, need


class _LinearActGrad(torch.autograd.Function):
    """linear_act_f8 with linear_act_f8_backward as its gradient; `saved` receives what the latter reads."""

    @staticmethod
    def forward(ctx, X, W, bias, residual, act, sync, ws, saved):
        Y, (kept, *ctx.rest) = linear_act_f8(X, W, bias, act, residual, sync, ws)
        ctx.save_for_backward(kept)
        ctx.call = sync, W.dtype, ws
        saved.extend((kept, *ctx.rest))
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        _check_capture("linear_act_f8", ctx)
        *needs, residual = ctx.needs_input_grad[:4]
        grads = linear_act_f8_backward(dY, (*ctx.saved_tensors, *ctx.rest), *ctx.call, *needs) if any(needs) else (None,) * 3
        return *grads, dY if residual else None, None, None, None, None


def linear_act_f8(X: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, act: str | None = None,
                  residual: torch.Tensor | None = None, sync: bool = True, ws: torch.Tensor | None = None):
    """(Y, saved): Y = act(X W^T + bias) + residual, with X [M, K] and W [N, K] quantised as in linear_f8, in X's
    dtype, which residual [M, N] has too; bias [N].  `saved` is what linear_act_f8_backward needs: with an
    activation also X W^T + bias in X's dtype, where the activation's slope is taken.  Where an argument requires a
    gradient autograd calls linear_act_f8_backward for Y."""
    if _differentiable(X, W, X, W, bias, residual):
        saved = []
        return _LinearActGrad.apply(X, W, bias, residual, act, sync, ws, saved), tuple(saved)
    where = "linear_act_f8"
    a = _act(where, act)
    if ws is None and X.is_cuda:
        r = _native().linear_act(X, W, bias, a, residual, RG_FLAG_SYNC if sync else 0)
        if r is not None:
            Y, kept, M, N, K = r
            return Y, (kept, M, N, K, act, X.dtype, None if bias is None else bias.dtype)
    tx, tw = _TYPES.get(X.dtype), _TYPES.get(W.dtype)
    if tx is None or tw is None or X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[1] or not X.shape[1]:
        raise ValueError(f"{where}: X [M, K] and W [N, K] float32, float16 or bfloat16 expected")
    idx = _device_index(where, X, W, *_there(bias, residual))
    (M, K), N = X.shape, W.shape[0]
    bias, tb, residual, ldr = _beside(where, M, N, bias, residual, X.dtype)
    nsaved, need = _linear_act_bytes(M, N, K, tx, a)
    X, ldx = _rows_of(X)
    W, ldw = _rows_of(W)
    Y = torch.empty((M, N), dtype=X.dtype, device=X.device)
    kept = torch.empty(nsaved, dtype=torch.uint8, device=X.device)
    w = ws if ws is not None else _scratch(need, idx)
    _launch(idx, where, library().linear_act_f8, X.data_ptr(), tx, ldx, W.data_ptr(), tw, ldw, _ptr(bias), tb, a,
            _ptr(residual), ldr, Y.data_ptr(), M, N, K, kept.data_ptr(), nsaved, RG_FLAG_SYNC if sync else 0,
            w.data_ptr(), w.numel())
    return Y, (kept, M, N, K, act, X.dtype, None if bias is None else bias.dtype)


def linear_act_f8_backward(dY: torch.Tensor, saved, sync: bool = True, dw_dtype: torch.dtype = torch.float32,
                           ws: torch.Tensor | None = None, dx: bool = True, dw: bool = True, db: bool = True):
    """(dX, dW, dbias) of linear_act_f8 for the output's gradient dY [M, N], in the output's dtype: with d = dY times
    the activation's slope (float32), dX = d W and dW = d^T X, with d quantised along N and along M, dX in dY's dtype,
    dW in dw_dtype, and dbias = the sum of d's rows in bias's dtype (None without a bias).  The residual's gradient is
    dY.  With dx, dw or db false that gradient is not computed, and None."""
    kept, M, N, K, act, dtype, bias_dtype = saved
    where = "linear_act_f8_backward"
    t, tw = _TYPES.get(dY.dtype), _TYPES.get(dw_dtype)
    if dY.dtype != dtype or tw is None or dY.shape != (M, N):
        raise ValueError(f"{where}: dY with the output's shape and dtype expected")
    a = _act(where, act)
    if not db:
        bias_dtype = None
    flags = _backward_flags(sync, dx, dw)
    if ws is None and dY.is_cuda:
        r = _native().linear_act_backward(dY, kept, M, N, K, a, bias_dtype, dw_dtype, flags)
        if r is not None:
            return r
    idx = _device_index(where, dY, kept)
    need = _linear_act_bytes(M, N, K, t, a)[1]
    dY, lddy = _rows_of(dY)
    dX = torch.empty((M, K), dtype=dtype, device=dY.device) if dx else None
    dW = torch.empty((N, K), dtype=dw_dtype, device=dY.device) if dw else None
    dbias = None if bias_dtype is None else torch.empty(N, dtype=bias_dtype, device=dY.device)
    w = ws if ws is not None else _scratch(need, idx)
    _launch(idx, where, library().linear_act_f8_backward, dY.data_ptr(), t, lddy, kept.data_ptr(), kept.numel(), a,
            _ptr(dX), _ptr(dW), tw, _ptr(dbias), _TYPES.get(bias_dtype, 0), M, N, K, flags, w.data_ptr(), w.numel())
    return dX, dW, dbias
