"""8-bit products with bias, activation and residual against plain 64-bit implementations.

Bounds, with u the unit roundoff of the result's format:

p         as in test_gpu_f8.py, |error| <= e_p = (144 + KB) 2^-23 sum |a b|, and 2^-24 of each sum with the bias
act(p)    every activation's slope is within (-0.2, 1.2), so e_p counts at most 1.2 times.  Its own evaluation: an
          exponential of relative error 2^-22 (its argument carries up to three roundings, |argument| e^argument /
          (1 + e^argument)^2 < 1/4 of which reach the result, times at most 2), the quotient 2^-22, the products
          2^-23; 1 + erf(x / sqrt 2) is off by up to 2^-22 in absolute terms.  Together at most |p| 2^-20.
slope     sums of at most three such terms, each at most (1 + |p|): (1 + |p|) 2^-19
d         |dy| (1 + |p|) 2^-19.  Quantised, an entry within that of a border between two E4M3 values may fall to the
          other side: one step of its value there, counted for those entries alone.
"""
import math

import numpy as np
import pytest
import torch

from gpu_util import rg, variant  # noqa: F401
from test_gpu_f8 import GRID, U, block_max, blocks, normal, quantise_reference, random_f8, random_scales, spread

pytestmark = pytest.mark.gpu

ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]
erf = np.vectorize(math.erf)


def act64(x, act):
    with np.errstate(over="ignore"):
        if act == "relu":
            return np.maximum(x, 0)
        if act == "silu":
            return x / (1 + np.exp(-x))
        if act == "gelu":
            return x * (1 + erf(x / math.sqrt(2))) / 2
        if act == "gelu_tanh":
            return x * (1 + np.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x**3))) / 2
    return x


def slope64(x, act):
    if act == "relu":
        return (x > 0).astype(float)
    if act is None:
        return np.ones_like(x)
    if act == "gelu":
        return (1 + erf(x / math.sqrt(2))) / 2 + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    with np.errstate(over="ignore"):
        if act == "silu":
            s = 1 / (1 + np.exp(-x))
            return s * (1 + x * (1 - s))
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (x + 0.044715 * x**3))
        return (1 + t) / 2 + x * (1 - t * t) * c * (1 + 0.134145 * x * x) / 2


def operands(m, n, k, seed):
    A, a = random_f8(m, k, seed + 1)
    B, b = random_f8(n, k, seed + 2)
    SA, sa = random_scales((m, blocks(k)), seed + 3)
    SB, sb = random_scales((blocks(n), blocks(k)), seed + 4)
    SA, sa = SA * 2.0**-8, sa * 2.0**-8  # p of the order of 1
    SB, sb = SB * 2.0**-8, sb * 2.0**-8
    av, bv = a * spread(sa, 1, 128, a.shape), b * spread(sb, 128, 128, b.shape)
    return (A, SA, B, SB), av @ bv.T, (144 + blocks(k)) * 2.0**-23 * (np.abs(av) @ np.abs(bv).T)


def within(got, ref, bound):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], bound[bad][:5])


def check_product(rg, m, n, k, act, out, bias, residual, pre, seed=0):  # noqa: F811
    args, p, ep = operands(m, n, k, seed)
    b = normal((n,), seed + 5, 0.5, bias) if bias else None
    r = normal((m, n), seed + 6, 1.0, out) if residual else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = rg.scaled_gemm_act_f8(*args, bias=dev(b), act=act, residual=dev(r), pre=pre, out_dtype=out)
    C, P = got if pre else (got, None)
    assert C.shape == (m, n) and C.dtype == out
    if bias:
        p = p + b.double().numpy()
        ep = ep + 2.0**-24 * np.abs(p)
    tiny = 2.0**-25 if out == torch.float16 else 0
    if pre:
        within(P, p, ep + U[out] * np.abs(p) + tiny)
    y = act64(p, act)
    ey = 1.2 * ep + (np.abs(p) * 2.0**-20 if act not in (None, "relu") else 0)
    if residual:
        y = y + r.double().numpy()
        ey = ey + 2.0**-24 * np.abs(y)
    within(C, y, ey + U[out] * (np.abs(y) + ey) + tiny)
    return C


SHAPES = [(1, 1, 1), (1, 300, 2000), (7, 33, 65), (17, 1000, 1024), (30, 129, 257), (64, 64, 4096), (130, 260, 1000),
          (300, 512, 127), (1000, 776, 520)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(rg, m, n, k, act):  # noqa: F811
    check_product(rg, m, n, k, act, torch.float32, torch.float32, True, True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (130, 264, 1000), (257, 513, 200)])
def test_product_kernels(rg, variant, m, n, k, out, act):  # noqa: F811
    """Both tensor-core kernels, whatever the shape would choose, with and without each part of the epilogue."""
    for i, bias in enumerate((None, torch.float32, torch.bfloat16, torch.float16)):
        check_product(rg, m, n, k, act, out, bias, i % 2 == 0, i < 2, seed=30 + i)


@pytest.mark.parametrize("m,n,k,out", [(4, 4096, 512, torch.bfloat16), (16, 2048, 300, torch.float16),
                                       (24, 520, 1024, torch.bfloat16), (32, 511, 640, torch.bfloat16),
                                       (200, 4104, 264, torch.float16), (2100, 2300, 640, torch.bfloat16),
                                       (2048, 2304, 384, torch.float32)])
def test_product_sizes(rg, m, n, k, out):  # noqa: F811
    for act, residual in (("silu", True), (None, True), ("gelu", False)):
        check_product(rg, m, n, k, act, out, out, residual, act == "gelu", seed=60)


def test_product_without_epilogue_is_the_plain_one(rg):  # noqa: F811
    for m in (3, 20, 200, 2100):
        args, _, _ = operands(m, 2304, 260, 1)
        want = rg.scaled_gemm_f8(*args, transb=True)
        assert torch.equal(rg.scaled_gemm_act_f8(*args), want)
        assert torch.equal(rg.scaled_gemm_act_f8(*args, act="silu", pre=True)[1], want)


@pytest.mark.parametrize("m", [5, 300, 2100])
def test_product_strides_alignment_and_out(rg, m):  # noqa: F811
    n = 2080
    args, _, _ = operands(m, n, 260, 1)
    bias = normal((2 * n,), 2).cuda()[::2]
    wide = normal((m, n + 30), 3, 1.0, torch.bfloat16).cuda()
    for r in (wide[:, :n], wide[:, 1 : n + 1], wide[:, 8 : n + 8], wide[:, :n].t().contiguous().t(),
              wide[:1, :n].expand(m, n)):
        want = rg.scaled_gemm_act_f8(*args, bias=bias.contiguous(), act="silu", residual=r.clone(
            memory_format=torch.contiguous_format))
        assert torch.equal(rg.scaled_gemm_act_f8(*args, bias=bias, act="silu", residual=r), want)
        buf = torch.full((m * n + 2,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[1:-1].view(m, n)  # off 16-byte boundaries
        assert rg.scaled_gemm_act_f8(*args, bias=bias, act="silu", residual=r, out=out) is out
        assert torch.equal(out, want) and buf[0] == 7 and buf[-1] == 7
    # in place of the residual
    r = wide[:, :n].contiguous()
    want = rg.scaled_gemm_act_f8(*args, bias=bias, act="gelu", residual=r)
    for _ in range(5):
        again = r.clone()
        rg.scaled_gemm_act_f8(*args, bias=bias, act="gelu", residual=again, out=again)
        assert torch.equal(again, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [512, 508, 506, 505, 490, 264])
def test_product_on_every_boundary(rg, variant, n, dtype):  # noqa: F811
    """Results and a residual whose rows start 0, 1, 2, 4 entries off 16-byte boundaries: bits as on them, and nothing
    written beside the result."""
    m, k = 300, 520
    (A, SA, B, SB), _, _ = operands(m, 512, k, 3)
    bias, r = normal((512,), 4, 0.5, dtype).cuda(), normal((m, 512), 5, 1.0, dtype).cuda()
    want, first = rg.scaled_gemm_act_f8(A, SA, B, SB, bias, "gelu", r, True, dtype)
    product = rg.scaled_gemm_f8(A, SA, B, SB, dtype, True)
    B = B[:n].contiguous()
    SB = SB[: blocks(n)].contiguous()
    wide = torch.empty((m, n + 8 + 8 - n % 8), dtype=dtype, device="cuda")
    for off in (0, 1, 2, 4):
        res = wide[:, off : off + n]
        res.copy_(r[:, :n])
        buf = torch.full((m * n + 16,), 7.0, dtype=dtype, device="cuda")
        out = buf[off : off + m * n].view(m, n)
        for bound in (res, res.contiguous()):
            _, p = rg.scaled_gemm_act_f8(A, SA, B, SB, bias[:n], "gelu", bound, True, out=out, out_dtype=dtype)
            assert torch.equal(out, want[:, :n]) and torch.equal(p, first[:, :n])
            assert (buf[:off] == 7).all() and (buf[off + m * n :] == 7).all()
            buf[off : off + m * n] = 7
        own = buf[off : off + m * n].view(m, n)
        own.copy_(r[:, :n])  # in the residual's place
        rg.scaled_gemm_act_f8(A, SA, B, SB, bias[:n], "gelu", own, out=own, out_dtype=dtype)
        assert torch.equal(own, want[:, :n])
        assert (buf[:off] == 7).all() and (buf[off + m * n :] == 7).all()
        rg.scaled_gemm_f8(A, SA, B, SB, dtype, True, out=own)
        assert torch.equal(own, product[:, :n])
        assert (buf[:off] == 7).all() and (buf[off + m * n :] == 7).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 40, 300])
def test_special_values(rg, variant, act, m):  # noqa: F811
    """Large, infinite and NaN values before the activation: what the formula gives, and in their own column alone.
    The operands are zeros, so that p is the bias."""
    vals = [0.0, -0.0, 1e-30, -1e-30, 0.7, -0.7, 12.0, -12.0, 40.0, -40.0, 90.0, -90.0, 150.0, -150.0, 1e10, -1e10,
            1e20, -1e20, 3e38, -3e38, math.inf, math.nan]
    bias = torch.tensor(vals * 13, device="cuda")
    n = bias.numel()
    A, B = (torch.zeros(s, device="cuda").to(torch.float8_e4m3fn) for s in ((m, 64), (n, 64)))
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    C, P = rg.scaled_gemm_act_f8(A, one(m, 1), B, one(blocks(n), 1), bias=bias, act=act, pre=True,
                                 out_dtype=torch.float32)
    x = bias.double().cpu().numpy()
    assert torch.equal(P.isnan(), bias.isnan().expand(m, n)) and torch.equal(P.nan_to_num(), bias.nan_to_num().expand(m, n))
    with np.errstate(over="ignore", invalid="ignore"):
        ref = act64(x, act)
    got = C.double().cpu().numpy()
    assert (np.isnan(got) == np.isnan(ref)).all()
    fine = np.isfinite(ref)
    assert (got[:, np.isinf(ref)] == ref[np.isinf(ref)]).all()
    tol = np.minimum(np.abs(x[fine]), 200) * 2.0**-20 + 2.0**-23 * np.abs(ref[fine]) + 2.0**-126
    if act in (None, "relu"):
        tol[:] = 0
    assert (np.abs(got[:, fine] - ref[fine]) <= tol).all()


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------


def layer_inputs(m, n, k, dtype, seed=0, scale=2.0):
    x, w = normal((m, k), seed + 1, scale, dtype), normal((n, k), seed + 2, k**-0.5, torch.bfloat16).float()
    return x.cuda(), w.cuda(), normal((n,), seed + 3, 0.5, dtype).cuda(), normal((m, n), seed + 4, 2.0**-4, dtype).cuda()


def uncertain(d, e):
    """(d quantised along its rows, how far that may be off for entries that may be off by e)"""
    q, s = quantise_reference(d, 1)
    a = np.maximum(block_max(d, 1, 128), 2.0**-60)
    rel = spread(block_max(e, 1, 128) / a, 1, 128, d.shape) + 2.0**-22  # of the scale
    s = spread(s, 1, 128, d.shape)
    v, top = np.abs(d) / s, np.abs(q)
    i = np.searchsorted(GRID, top)
    up, down = GRID[(i + 1).clip(0, 126)] - top, top - GRID[(i - 1).clip(0, 126)]
    near = np.minimum(np.abs(v - (top + up / 2)), np.abs(v - (top - down / 2))) <= e / s + v * rel
    return q * s, np.where(near, np.maximum(up, down) * s, 0) + np.abs(q) * s * rel


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k,dtype", [(1, 130, 200, torch.bfloat16), (200, 136, 264, torch.bfloat16),
                                         (131, 257, 129, torch.float16), (300, 150, 70, torch.float32)])
def test_layer_gradients(rg, m, n, k, dtype, act):  # noqa: F811
    x, w, b, dy = layer_inputs(m, n, k, torch.bfloat16 if dtype == torch.float32 else dtype)
    x, b, dy = x.to(dtype), b.to(dtype), dy.to(dtype)
    Y, saved = rg.linear_act_f8(x, w, bias=b, act=act)
    dX, dW, db = rg.linear_act_f8_backward(dy, saved)
    assert Y.dtype == dX.dtype == db.dtype == dtype and dW.dtype == torch.float32 and db.shape == (n,)
    # p as it is kept (test_layer_is_its_parts shows that this is it)
    qx, sx = rg.quantize_f8(x)
    qw, sw = rg.quantize_f8(w, "tiles")
    want, P = rg.scaled_gemm_act_f8(qx, sx, qw, sw, bias=b, act=act, pre=True, out_dtype=dtype)
    assert torch.equal(Y, want)
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    p, dd, xd = host(P), host(dy), host(x)
    d, e = dd * slope64(p, act), np.abs(dd) * (1 + np.abs(p)) * 2.0**-19
    if act in (None, "relu"):
        e = np.zeros_like(d)
    wv = host(qw) * spread(host(sw), 128, 128, w.shape)
    q, s = quantise_reference(xd.T, 1)
    xv = q * spread(s, 1, 128, xd.T.shape)
    for got, (a, ea), v in ((dX, uncertain(d, e), wv), (dW, uncertain(d.T, e.T), xv.T)):
        ref, mag = a @ v, np.abs(a) @ np.abs(v)
        within(got, ref, (146 + blocks(a.shape[1])) * 2.0**-23 * mag + ea @ np.abs(v) * 1.01 + U[got.dtype] * np.abs(ref)
               + 2.0**-24)
    ref = d.sum(0)
    # fp32 sums of m terms, at most m / 8 + 24 roundings in a row
    within(db, ref, e.sum(0) + (m / 8 + 24) * 2.0**-24 * np.abs(d).sum(0) + U[dtype] * np.abs(ref) * 1.01 + 2.0**-25)


@pytest.mark.parametrize("act", ACTS)
def test_slopes_against_differences(rg, act):  # noqa: F811
    """One row of zeros and the bias as p: dbias is dy times the slope there, against differences of the activation in
    64 bits (h = 2^-10: off by at most h^2 / 6 times its third derivative, below 2)."""
    b = torch.linspace(-14, 14, 1001, device="cuda")
    if act == "relu":
        b = b[b.abs() > 2.0**-9]
    x, w = torch.zeros((1, 40), device="cuda"), torch.ones((b.numel(), 40), device="cuda")
    Y, saved = rg.linear_act_f8(x, w, bias=b, act=act)
    dy = normal((1, b.numel()), 1).cuda()
    db = rg.linear_act_f8_backward(dy, saved)[2]
    p, h = b.double().cpu().numpy(), 2.0**-10
    slope = (act64(p + h, act) - act64(p - h, act)) / (2 * h)
    v = np.abs(dy[0].double().cpu().numpy())
    within(db, dy[0].double().cpu().numpy() * slope, v * ((1 + np.abs(p)) * 2.0**-19 + h * h / 3 + 2.0**-24 + 2.0**-40 / h))
    within(Y[0], act64(p, act), np.abs(p) * 2.0**-20)


@pytest.mark.parametrize("dtype,dw", [(torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16),
                                      (torch.float32, torch.float16)])
@pytest.mark.parametrize("m,act", [(70, None), (300, "relu"), (1, "relu"), (2100, "relu"), (300, None)])
def test_layer_is_its_parts(rg, m, act, dtype, dw):  # noqa: F811
    """With slopes of 0 and 1 the calls give what quantisation and products give one after the other, to the bit."""
    x = normal((m, 270), 1, 1.0, dtype).cuda()[:, 5:261]
    w = normal((256, 200), 2, 0.1).cuda().t()  # [200, 256], columns contiguous
    b, r = normal((200,), 3, 0.5).cuda(), normal((m, 210), 5, 1.0, dtype).cuda()[:, 3:203]
    dy = normal((m, 400), 4, 0.01, dtype).cuda()[:, ::2]
    Y, saved = rg.linear_act_f8(x, w, bias=b, act=act, residual=r)
    dX, dW, db = rg.linear_act_f8_backward(dy, saved, dw_dtype=dw)
    qx, sx, qxt, sxt = rg.quantize_f8(x, "both")
    qw, sw = rg.quantize_f8(w, "tiles")
    want, P = rg.scaled_gemm_act_f8(qx, sx, qw, sw, bias=b, act=act, residual=r, pre=True, out_dtype=dtype)
    assert torch.equal(Y, want) and db.dtype == torch.float32
    d = dy * (P > 0) if act else dy
    qd, sd, qdt, sdt = rg.quantize_f8(d, "both")
    assert torch.equal(dX, rg.scaled_gemm_f8(qd, sd, qw, sw, out_dtype=dtype))
    assert torch.equal(dW, rg.scaled_gemm_f8(qdt, sdt, qxt, sxt, transb=True, out_dtype=dw))
    assert (db - d.double().sum(0)).abs().max() <= (m / 8 + 24) * 2.0**-24 * d.double().abs().sum(0).max()
    # without a bias: no gradient for it
    Y, saved = rg.linear_act_f8(x, w, act=act)
    dX, dW, db = rg.linear_act_f8_backward(dy, saved, dw_dtype=dw)
    assert db is None
    if act is None:
        Y2, saved2 = rg.linear_f8(x, w)
        assert torch.equal(Y, Y2)
        assert all(torch.equal(p, q) for p, q in zip((dX, dW), rg.linear_f8_backward(dy, saved2, dw_dtype=dw)))


@pytest.mark.parametrize("act", [None, "gelu"])
def test_layer_has_a_gradient(rg, act):  # noqa: F811
    bf = torch.bfloat16
    x, w, b, dy = layer_inputs(70, 96, 200, bf)
    r = normal((70, 96), 9, 1.0, bf).cuda()
    want, saved = rg.linear_act_f8(x, w, bias=b, act=act, residual=r)
    grads = (*rg.linear_act_f8_backward(dy, saved), dy)
    for needs in ((1, 1, 1, 1), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1)):
        ts = [t.clone().requires_grad_(bool(n)) for t, n in zip((x, w, b, r), needs)]
        y, _ = rg.linear_act_f8(ts[0], ts[1], ts[2], act, ts[3], sync=False)
        assert y.requires_grad and torch.equal(y, want)
        y.backward(dy)
        for t, n, g in zip(ts, needs, grads):
            assert (t.grad is not None) == bool(n) and (not n or (t.grad.dtype == t.dtype and torch.equal(t.grad, g)))
    w1 = w.clone().requires_grad_()
    y, _ = rg.linear_act_f8(x, w1, act=act)  # neither bias nor residual
    (g,) = torch.autograd.grad(y.sum(), w1)
    _, saved = rg.linear_act_f8(x, w, act=act)
    assert torch.equal(g, rg.linear_act_f8_backward(torch.ones_like(y), saved)[1])


def test_product_without_a_gradient_does_not_cut_it_silently(rg):  # noqa: F811
    args, _, _ = operands(5, 96, 256, 1)
    b = torch.ones(96, device="cuda", requires_grad=True)
    for pre in (False, True):
        y = rg.scaled_gemm_act_f8(*args, bias=b, pre=pre)
        y = y[1] if pre else y
        assert y.requires_grad
        with pytest.raises(NotImplementedError):
            y.sum().backward()
    with pytest.raises(ValueError):
        rg.scaled_gemm_act_f8(*args, bias=b, out=torch.empty((5, 96), dtype=torch.bfloat16, device="cuda"))


def test_layer_saved_buffer_is_checked(rg):  # noqa: F811
    x, w, b, dy = layer_inputs(70, 96, 200, torch.bfloat16)
    _, (kept, *rest) = rg.linear_act_f8(x, w, bias=b, act="silu")
    with pytest.raises(rg.ResGemmError) as err:
        rg.linear_act_f8_backward(dy, (kept[:-256], *rest))
    assert err.value.code == rg.RG_ERR_WORKSPACE
    for bad, dw in ((dy[:, :-1], torch.float32), (dy[:-1], torch.float32), (dy.float(), torch.float32), (dy, torch.float64)):
        with pytest.raises(ValueError):
            rg.linear_act_f8_backward(bad, (kept, *rest), dw_dtype=dw)


def test_empty(rg):  # noqa: F811
    e = lambda *s: torch.zeros(s, device="cuda").to(torch.float8_e4m3fn)  # noqa: E731
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    assert rg.scaled_gemm_act_f8(e(0, 7), one(0, 1), e(5, 7), one(1, 1), bias=one(5), act="silu").shape == (0, 5)
    x, w = one(0, 40), one(30, 40)
    Y, saved = rg.linear_act_f8(x, w, bias=one(30), act="gelu", residual=one(0, 30))
    dX, dW, db = rg.linear_act_f8_backward(Y, saved)
    assert Y.shape == (0, 30) and dX.shape == (0, 40) and (dW == 0).all() and (db == 0).all() and db.shape == (30,)


def test_timeout_is_reported(rg, variant):  # noqa: F811
    lib = rg.library()
    args, _, _ = operands(512, 512, 512, 1)
    b = torch.ones(512, device="cuda")
    good = rg.scaled_gemm_act_f8(*args, bias=b, act="silu")
    old = lib.rg_set_wait_limit_ns(50_000_000)
    try:
        lib.rg_inject_fault(1)
        with pytest.raises(rg.ResGemmError) as err:
            rg.scaled_gemm_act_f8(*args, bias=b, act="silu")
        assert err.value.code == rg.RG_ERR_TIMEOUT
    finally:
        lib.rg_inject_fault(0)
        lib.rg_set_wait_limit_ns(old)
    assert torch.equal(rg.scaled_gemm_act_f8(*args, bias=b, act="silu"), good)


def test_product_of_many_entries(rg):  # noqa: F811
    """Results, residual and values before the activation whose entries pass 2^31."""
    m, n = 70000, 32768
    A, a = random_f8(m, 16, 1)
    B, b = random_f8(n, 16, 2)
    SA, sa = random_scales((m, 1), 3)
    SB, sb = random_scales((n // 128, 1), 4)
    r = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    r[::7] = 1.0
    C, P = rg.scaled_gemm_act_f8(A, SA, B, SB, act="relu", residual=r, pre=True)
    bv = b * np.repeat(sb, 128, 0)
    for row in (0, 7, 65535, 65536, 69993, 69999):
        av = a[row] * sa[row]
        ref, e = bv @ av, 145 * 2.0**-23 * (np.abs(bv) @ np.abs(av))
        within(P[row], ref, e + U[torch.bfloat16] * np.abs(ref))
        y = np.maximum(ref, 0) + (row % 7 == 0)
        within(C[row], y, e + 2.0**-24 * np.abs(y) + U[torch.bfloat16] * (np.abs(y) + e))
