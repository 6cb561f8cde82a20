"""What the 8-bit products by group and with an epilogue refuse, before any device work (no GPU)."""
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


def test_product_with_epilogue_arguments(rg, mem):
    p, f = mem[0], rg.library().scaled_gemm_act_f8

    def call(A=p, lda=16, SA=p, B=p, ldb=16, SB=p, bias=p, bt=0, act=2, R=p, ldr=8, P=p, C=p, ct=2, ldc=8, M=4, N=8,
             K=16, ws=p, wsb=4096):
        return f(A, lda, SA, B, ldb, SB, bias, bt, act, R, ldr, P, C, ct, ldc, M, N, K, 0, ws, wsb, None)

    for bad in (dict(A=None), dict(SA=None), dict(B=None), dict(SB=None), dict(C=None), dict(ct=3), dict(bt=3),
                dict(bt=-1), dict(act=-1), dict(act=5), dict(ldr=7), dict(lda=15), dict(lda=24), dict(ldb=8),
                dict(A=p + 8), dict(B=p + 1), dict(ldc=7), dict(M=-1), dict(N=-1), dict(K=0), dict(K=-2), dict(M=2**31),
                dict(N=2**40), dict(ws=None), dict(ws=p + 16), dict(M=2**30, N=2**30, ldc=2**30, ldr=2**30)):
        assert call(**bad) == rg.RG_ERR_ARG, bad
    assert call(wsb=4095) == rg.RG_ERR_WORKSPACE


def test_layer_with_epilogue_arguments(rg, mem):
    p, lib = mem[0], rg.library()
    saved, need = lib.linear_act_f8_saved_bytes(4, 8, 16, 2, 2), lib.linear_act_f8_ws_bytes(4, 8, 16)
    assert saved > lib.linear_act_f8_saved_bytes(4, 8, 16, 2, 0) > 0 and need > 4096
    for bad in ((-1, 8, 16), (2**31, 8, 16), (4, 8, 0), (2**30, 2**30, 16)):
        assert lib.linear_act_f8_ws_bytes(*bad) == 0 and lib.linear_act_f8_saved_bytes(*bad, 2, 1) == 0
    assert lib.linear_act_f8_saved_bytes(4, 8, 16, 3, 1) == 0 and lib.linear_act_f8_saved_bytes(4, 8, 16, 2, 5) == 0

    def forward(X=p, xt=2, ldx=16, W=p, wt=0, ldw=16, bias=p, bt=1, act=2, R=p, ldr=8, Y=p, M=4, N=8, K=16, sv=p,
                svb=saved, ws=p, wsb=need):
        return lib.linear_act_f8(X, xt, ldx, W, wt, ldw, bias, bt, act, R, ldr, Y, M, N, K, sv, svb, 0, ws, wsb, None)

    def backward(dY=p, t=2, ld=8, sv=p, svb=saved, act=2, dX=p, dW=p, wt=0, db=p, bt=0, M=4, N=8, K=16, ws=p, wsb=need):
        return lib.linear_act_f8_backward(dY, t, ld, sv, svb, act, dX, dW, wt, db, bt, M, N, K, 0, ws, wsb, None)

    for bad in (dict(X=None), dict(W=None), dict(Y=None), dict(xt=3), dict(wt=-1), dict(bt=3), dict(act=5), dict(ldx=15),
                dict(ldw=15), dict(ldr=7), dict(M=-1), dict(N=2**31), dict(K=0), dict(sv=None), dict(sv=p + 16),
                dict(ws=None), dict(ws=p + 16)):
        assert forward(**bad) == rg.RG_ERR_ARG, bad
    for bad in (dict(dY=None), dict(dX=None), dict(dW=None), dict(t=3), dict(wt=3), dict(bt=3), dict(act=-1), dict(ld=7),
                dict(K=0), dict(sv=None), dict(sv=p + 128), dict(ws=None)):
        assert backward(**bad) == rg.RG_ERR_ARG, bad
    for f in (forward, backward):
        assert f(wsb=need - 1) == rg.RG_ERR_WORKSPACE and f(svb=saved - 1) == rg.RG_ERR_WORKSPACE


def test_quantisation_by_group_arguments(rg, mem):
    p, f = mem[0], rg.library().quantize_grouped_f8

    def call(x=p, xt=0, ldx=8, M=4, K=8, form=2, off=p, E=2, q=p, ldq=8, s=p, qt=p, ldqt=256, st=p, flags=0):
        return f(x, xt, ldx, M, K, form, off, E, q, ldq, s, qt, ldqt, st, flags, None)

    for bad in (dict(x=None), dict(xt=3), dict(ldx=7), dict(M=-1), dict(K=-1), dict(M=2**31), dict(form=0), dict(form=4),
                dict(off=None), dict(off=p + 2), dict(off=p + 4, flags=16), dict(E=0), dict(E=513), dict(q=None),
                dict(s=None), dict(ldq=7), dict(qt=None), dict(st=None), dict(ldqt=255), dict(form=1, qt=None),
                dict(form=3, q=None), dict(form=3, E=0), dict(form=3, ldx=7), dict(form=3, s=None),
                dict(M=2**30, K=2**30, ldx=2**30, ldq=2**30, ldqt=2**31)):
        assert call(**bad) == rg.RG_ERR_ARG, bad


def test_product_by_group_arguments(rg, mem):
    p, lib = mem[0], rg.library()

    def rows(A=p, lda=16, SA=p, B=p, ldb=16, SB=p, off=p, E=2, C=p, ct=2, ldc=8, T=4, N=8, K=16, flags=4, ws=p,
             wsb=4096):
        return lib.grouped_gemm_f8(A, lda, SA, B, ldb, SB, off, E, C, ct, ldc, T, N, K, flags, ws, wsb, None)

    def sums(A=p, lda=256, SA=p, B=p, ldb=256, SB=p, off=p, E=2, C=p, ct=0, M=4, N=8, nb=2, flags=0, ws=p, wsb=4096):
        return lib.grouped_wgrad_f8(A, lda, SA, B, ldb, SB, off, E, C, ct, M, N, nb, flags, ws, wsb, None)

    both = (dict(A=None), dict(SA=None), dict(B=None), dict(SB=None), dict(C=None), dict(ct=3), dict(off=None),
            dict(off=p + 1), dict(off=p + 4, flags=20), dict(E=0), dict(E=-1), dict(E=513), dict(lda=15), dict(lda=24),
            dict(ldb=8), dict(A=p + 8), dict(B=p + 1), dict(N=-1), dict(N=2**40), dict(ws=None), dict(ws=p + 16))
    for bad in (*both, dict(ldc=7), dict(T=-1), dict(K=0), dict(K=2**31), dict(T=2**31), dict(flags=0, ldb=0),
                dict(T=2**30, N=2**30, ldc=2**30)):
        assert rows(**bad) == rg.RG_ERR_ARG, bad
    for bad in (*both, dict(M=-1), dict(nb=1), dict(nb=2**24, lda=2**31, ldb=2**31), dict(M=2**30), dict(lda=240)):
        assert sums(**bad) == rg.RG_ERR_ARG, bad
    assert rows(wsb=4095) == rg.RG_ERR_WORKSPACE and sums(wsb=4095) == rg.RG_ERR_WORKSPACE


def test_layer_by_group_arguments(rg, mem):
    p, lib = mem[0], rg.library()
    saved, need = lib.expert_linear_f8_saved_bytes(4, 8, 16, 2), lib.expert_linear_f8_ws_bytes(4, 8, 16, 2)
    assert saved > 0 and need > 4096
    for f in (lib.expert_linear_f8_saved_bytes, lib.expert_linear_f8_ws_bytes):
        for bad in ((-1, 8, 16, 2), (2**31, 8, 16, 2), (4, 8, 0, 2), (4, 8, 16, 0), (4, 8, 16, 513), (4, 2**22, 16, 512),
                    (2**30, 2**30, 16, 1)):
            assert f(*bad) == 0, bad

    def forward(X=p, xt=2, ldx=16, W=p, wt=0, ldw=16, off=p, E=2, Y=p, T=4, N=8, K=16, sv=p, svb=saved, ws=p, wsb=need):
        return lib.expert_linear_f8(X, xt, ldx, W, wt, ldw, off, E, Y, T, N, K, sv, svb, 0, ws, wsb, None)

    def backward(dY=p, t=2, ld=8, sv=p, svb=saved, off=p, E=2, dX=p, dW=p, wt=0, T=4, N=8, K=16, ws=p, wsb=need):
        return lib.expert_linear_f8_backward(dY, t, ld, sv, svb, off, E, dX, dW, wt, T, N, K, 0, ws, wsb, None)

    for bad in (dict(X=None), dict(W=None), dict(Y=None), dict(xt=3), dict(wt=-1), dict(ldx=15), dict(ldw=15),
                dict(off=None), dict(off=p + 1), dict(E=0), dict(T=-1), dict(N=2**31), dict(K=0), dict(sv=None),
                dict(sv=p + 16), dict(ws=None), dict(ws=p + 16)):
        assert forward(**bad) == rg.RG_ERR_ARG, bad
    for bad in (dict(dY=None), dict(dX=None), dict(dW=None), dict(t=3), dict(wt=3), dict(ld=7), dict(off=None),
                dict(E=513), dict(K=-1), dict(sv=None), dict(sv=p + 128), dict(ws=None)):
        assert backward(**bad) == rg.RG_ERR_ARG, bad
    for f in (forward, backward):
        assert f(wsb=need - 1) == rg.RG_ERR_WORKSPACE and f(svb=saved - 1) == rg.RG_ERR_WORKSPACE


def test_binding_refuses(rg):
    q = lambda *s: torch.zeros(s).to(F8)  # noqa: E731
    one, off = torch.ones, torch.zeros(3, dtype=torch.int32)
    x, w = torch.zeros((4, 200)), torch.zeros((2, 30, 200))
    act = lambda A=q(2, 200), SA=one(2, 2), B=q(3, 200), SB=one(1, 2), **kw: rg.scaled_gemm_act_f8(A, SA, B, SB, **kw)  # noqa: E731
    rows = lambda A=q(4, 200), SA=one(4, 2), B=q(2, 30, 200), SB=one(2, 1, 2), o=off, **kw: rg.grouped_gemm_f8(  # noqa: E731
        A, SA, B, SB, o, **{"transb": True, **kw})
    sums = lambda A=q(5, 256), SA=one(5, 2), B=q(6, 256), SB=one(6, 2), o=off, **kw: rg.grouped_wgrad_f8(  # noqa: E731
        A, SA, B, SB, o, **kw)
    for bad in (lambda: act(),  # not on a GPU, as the next to last of each
                lambda: act(act="swish"), lambda: act(bias=one(4)), lambda: act(bias=one(3).double()),
                lambda: act(residual=one(2, 3)), lambda: act(SB=one(3, 2)), lambda: act(SA=one(2, 1)),
                lambda: act(out_dtype=torch.float64), lambda: act(A=x), lambda: act(B=q(3, 199)),
                lambda: act(A=q(2, 0), SA=one(2, 0), B=q(3, 0), SB=one(1, 0)),
                lambda: rows(), lambda: rows(o=off.float()), lambda: rows(o=off[:2]), lambda: rows(o=off[None]),
                lambda: rows(SB=one(2, 2, 1)), lambda: rows(SA=one(4, 1)), lambda: rows(B=q(30, 200)),
                lambda: rows(transb=False), lambda: rows(out_dtype=torch.int32), lambda: rows(A=x),
                lambda: sums(), lambda: sums(o=off.to(torch.int16)), lambda: sums(o=torch.zeros(4, dtype=torch.int32)),
                lambda: sums(SA=one(5, 3)), lambda: sums(A=q(5, 128)), lambda: sums(A=q(5, 130), B=q(6, 130)),
                lambda: sums(out_dtype=torch.float64), lambda: rg.quantize_f8(x, "rows", offsets=off),
                lambda: rg.quantize_f8(x, "tiles", offsets=off), lambda: rg.quantize_f8(x, "both", offsets=off),
                lambda: rg.quantize_f8(x, "both", offsets=off.float()), lambda: rg.quantize_f8(w, "rows"),
                lambda: rg.quantize_f8(w, "tiles"), lambda: rg.quantize_f8(w.double(), "tiles"),
                lambda: rg.linear_act_f8(x, torch.zeros((3, 100))), lambda: rg.linear_act_f8(x, torch.zeros((3, 200))),
                lambda: rg.linear_act_f8(x, torch.zeros((3, 200)), act="tanh"),
                lambda: rg.expert_linear_f8(x, w[:, :, 1:], off), lambda: rg.expert_linear_f8(x, w, off),
                lambda: rg.expert_linear_f8(x, w, off[:2]), lambda: rg.expert_linear_f8(x.double(), w, off)):
        with pytest.raises(ValueError):
            bad()


def test_calls_wait_for_their_turn(rg, mem):
    """Calls without entries enqueue nothing but the clearing of the workspace's first words; they wait for its turn."""
    import threading

    lib, ws, other = rg.library(), mem[0], mem[0] + 32768
    big = 1 << 14
    calls = (lambda w: lib.scaled_gemm_act_f8(None, 16, None, None, 16, None, None, 0, 0, None, 0, None, None, 0, 4, 0, 4,
                                              16, 0, w, big, None),
             lambda w: lib.grouped_gemm_f8(None, 16, None, None, 16, None, other, 2, None, 0, 4, 0, 4, 16, 4, w, big, None),
             lambda w: lib.grouped_wgrad_f8(None, 256, None, None, 256, None, other, 2, None, 0, 0, 4, 2, 0, w, big, None),
             lambda w: lib.linear_act_f8(None, 0, 16, None, 0, 16, None, 0, 0, None, 0, None, 0, 0, 16, other, big, 0, w,
                                         big, None),
             lambda w: lib.linear_act_f8_backward(None, 0, 0, other, big, 0, None, None, 0, None, 0, 0, 0, 16, 0, w, big,
                                                  None))
    for f in calls:
        done = threading.Event()
        t = threading.Thread(target=lambda: (f(ws), done.set()))
        assert lib.rg_hold_workspace(ws, 1) == rg.RG_OK
        try:
            t.start()
            assert not done.wait(0.3)
        finally:
            assert lib.rg_hold_workspace(ws, 0) == rg.RG_OK
        assert done.wait(30)
        t.join()
