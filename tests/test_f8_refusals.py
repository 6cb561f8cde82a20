"""What the 8-bit block-scaled operators refuse, before any device work (no GPU)."""
import ctypes

import pytest
import torch

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def rg():
    from exact_modular_int8_gb300 import build as b

    b.build()
    import exact_modular_int8_gb300 as m

    return m


@pytest.fixture(scope="module")
def mem():
    """(a 256-byte aligned host address, the buffer): never dereferenced by a refused call."""
    buf = (ctypes.c_uint8 * 65536)()
    return (ctypes.addressof(buf) + 255) // 256 * 256, buf


def test_quantize_arguments(rg, mem):
    p, f = mem[0], rg.library().quantize_f8

    def call(x=p, xt=0, ldx=8, M=4, K=8, form=0, q=p, ldq=8, s=p, qt=p, ldqt=4, st=p):
        return f(x, xt, ldx, M, K, form, q, ldq, s, qt, ldqt, st, 0, None)

    for bad in (dict(x=None), dict(xt=3), dict(xt=-1), dict(ldx=7), dict(M=-1), dict(K=-1), dict(M=2**31),
                dict(K=2**30 + 1), dict(form=4), dict(form=-1), dict(q=None), dict(s=None), dict(ldq=7),
                dict(form=1, qt=None), dict(form=1, st=None), dict(form=2, ldqt=3), dict(form=2, q=None),
                dict(form=3, s=None), dict(M=2**30, K=2**30, ldx=2**30, ldq=2**30)):
        assert call(**bad) == rg.RG_ERR_ARG, bad


def test_product_arguments(rg, mem):
    p, f = mem[0], rg.library().scaled_gemm_f8

    def call(A=p, lda=16, SA=p, B=p, ldb=16, SB=p, C=p, ct=2, ldc=8, M=4, N=8, K=16, flags=4, ws=p, wsb=4096):
        return f(A, lda, SA, B, ldb, SB, C, ct, ldc, M, N, K, flags, ws, wsb, None)

    for bad in (dict(A=None), dict(SA=None), dict(B=None), dict(SB=None), dict(C=None), dict(ct=3), dict(lda=15),
                dict(lda=24), dict(ldb=8), dict(ldb=17), dict(A=p + 8), dict(B=p + 1), dict(ldc=7), dict(M=-1),
                dict(N=-1), dict(K=-2), dict(M=2**31), dict(N=2**40), dict(K=2**31), dict(ws=None), dict(ws=p + 16),
                dict(flags=0, ldb=0), dict(M=2**30, N=2**30, ldc=2**30)):
        assert call(**bad) == rg.RG_ERR_ARG, bad
    assert call(wsb=4095) == rg.RG_ERR_WORKSPACE


def test_linear_arguments(rg, mem):
    p, lib = mem[0], rg.library()
    saved, need = lib.linear_f8_saved_bytes(4, 8, 16), lib.linear_f8_ws_bytes(4, 8, 16)
    assert saved > 0 and need > 4096
    for f in (lib.linear_f8_saved_bytes, lib.linear_f8_ws_bytes):
        assert f(-1, 8, 16) == 0 and f(2**31, 8, 16) == 0 and f(2**30, 2**30, 16) == 0

    def forward(X=p, xt=2, ldx=16, W=p, wt=0, ldw=16, Y=p, M=4, N=8, K=16, sv=p, svb=saved, ws=p, wsb=need):
        return lib.linear_f8(X, xt, ldx, W, wt, ldw, Y, M, N, K, sv, svb, 0, ws, wsb, None)

    def backward(dY=p, t=2, ld=8, sv=p, svb=saved, dX=p, dW=p, wt=0, M=4, N=8, K=16, ws=p, wsb=need):
        return lib.linear_f8_backward(dY, t, ld, sv, svb, dX, dW, wt, M, N, K, 0, ws, wsb, None)

    for bad in (dict(X=None), dict(W=None), dict(Y=None), dict(xt=3), dict(wt=-1), dict(ldx=15), dict(ldw=15),
                dict(M=-1), dict(N=2**31), dict(sv=None), dict(sv=p + 16), dict(ws=None), dict(ws=p + 16)):
        assert forward(**bad) == rg.RG_ERR_ARG, bad
    for bad in (dict(dY=None), dict(dX=None), dict(dW=None), dict(t=3), dict(wt=3), dict(ld=7), dict(K=-1),
                dict(sv=None), dict(sv=p + 128), dict(ws=None)):
        assert backward(**bad) == rg.RG_ERR_ARG, bad
    for f in (forward, backward):
        assert f(wsb=need - 1) == rg.RG_ERR_WORKSPACE and f(svb=saved - 1) == rg.RG_ERR_WORKSPACE


def test_expert_layer_arguments(rg, mem):
    p, lib = mem[0], rg.library()

    def call(X=p, xt=2, WR=p, W13=p, S13=p, W2=p, S2=p, Y=p, T=2, H=32, I=16, E=4, k=2, ws=p, wsb=1 << 30):
        return lib.moe_layer_f8(X, xt, WR, W13, S13, W2, S2, Y, T, H, I, E, k, 1, 0, ws, wsb, None)

    for bad in (dict(X=None), dict(WR=None), dict(W13=None), dict(S13=None), dict(W2=None), dict(S2=None),
                dict(Y=None), dict(xt=0), dict(xt=3), dict(T=-1), dict(H=0), dict(H=24), dict(I=8), dict(I=40),
                dict(E=0), dict(E=513), dict(k=0), dict(k=5), dict(E=32, k=17), dict(H=2**20), dict(I=2**20),
                dict(X=p + 2), dict(W13=p + 4), dict(W2=p + 8), dict(Y=p + 2), dict(ws=None), dict(ws=p + 128)):
        assert call(**bad) == rg.RG_ERR_ARG, bad
    assert call(T=65) == rg.RG_ERR_RANGE
    need = lib.moe_layer_f8_ws_bytes(2, 32, 16, 4, 2)
    assert need > 4096
    assert call(wsb=need - 1) == rg.RG_ERR_WORKSPACE
    for bad in ((-1, 32, 16, 4, 2), (65, 32, 16, 4, 2), (1, 31, 16, 4, 2), (1, 32, 16, 4, 5), (1, 32, 0, 4, 2)):
        assert lib.moe_layer_f8_ws_bytes(*bad) == 0
    assert lib.moe_layer_f8_ws_bytes(0, 32, 16, 4, 2) == 4096


def test_binding_refuses(rg):
    q = lambda *s: torch.zeros(s).to(F8)  # noqa: E731
    one = torch.ones
    x = torch.zeros((4, 200))
    for bad in (lambda: rg.quantize_f8(x), lambda: rg.quantize_f8(x, "cols"), lambda: rg.quantize_f8(x.double()),
                lambda: rg.quantize_f8(x[0]), lambda: rg.scaled_gemm_f8(q(2, 200), one(2, 2), q(3, 200), one(1, 2)),
                lambda: rg.scaled_gemm_f8(q(2, 200), one(2, 2), q(3, 200), one(1, 2), transb=True),  # not on a GPU
                lambda: rg.scaled_gemm_f8(q(2, 200), one(2, 1), q(3, 200), one(1, 2), transb=True),
                lambda: rg.scaled_gemm_f8(q(2, 200), one(2, 2), q(3, 200), one(2, 2), transb=True),
                lambda: rg.scaled_gemm_f8(q(2, 200), one(2, 2).double(), q(3, 200), one(1, 2), transb=True),
                lambda: rg.scaled_gemm_f8(x, one(4, 2), q(3, 200), one(1, 2), transb=True),
                lambda: rg.scaled_gemm_f8(q(2, 200), one(2, 2), q(3, 200), one(1, 2), torch.float64, True),
                lambda: rg.linear_f8(x, torch.zeros((3, 100))), lambda: rg.linear_f8(x, torch.zeros((3, 200)))):
        with pytest.raises(ValueError):
            bad()


def test_expert_layer_binding_refuses(rg):
    bf = torch.bfloat16
    good = dict(X=torch.zeros((2, 32), dtype=bf), WR=torch.zeros((4, 32), dtype=bf),
                W13=torch.zeros((4, 32, 32)).to(F8), S13=torch.ones((4, 1, 1)), W2=torch.zeros((4, 32, 16)).to(F8),
                S2=torch.ones((4, 1, 1)))
    for name, bad in (("X", torch.zeros((2, 32))), ("X", torch.zeros(32, dtype=bf)), ("WR", torch.zeros((4, 32))),
                      ("WR", torch.zeros((5, 32), dtype=bf)), ("W13", torch.zeros((4, 32, 32))),
                      ("W13", torch.zeros((4, 16, 32)).to(F8)), ("S13", torch.ones((4, 1, 2))),
                      ("S2", torch.ones((4, 1, 1)).double()), ("W2", torch.zeros((4, 16, 16)).to(F8)),
                      ("X", good["X"])):  # the last: valid shapes, not on a GPU
        with pytest.raises(ValueError):
            rg.moe_layer_f8(**{**good, name: bad}, top_k=2)
