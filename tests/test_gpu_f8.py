"""The 8-bit block-scaled operators against plain 64-bit implementations of their formulas.

Bounds are derived from the arithmetic, with u the unit roundoff of the result's format:

product   E4M3 products are exact in fp32.  One MMA of K = 32 adds 32 of them to the accumulator with at least
          24-bit aligned operands: at most 33 units of 2^-23 of the largest, so four per block give 4 * 33; the
          scale product, the multiply-add per block and the joining of up to 8 slices add KB + 12.  Hence
          |error| <= (144 + KB) 2^-23 sum |a b| + u |c|.
experts   the same kind of count for each of the two products and first-order propagation through
          silu(a) u (|silu'| < 1.1), the fp16 rounding of h (2^-12 relative, 2^-27 of the row's largest), and the
          router (see _moe_reference).
"""
import math
import os
import sys

import numpy as np
import pytest
import torch

from gpu_util import rg, variant  # noqa: F401

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}
F8 = torch.float8_e4m3fn


def blocks(x):
    return -(-x // 128)


def normal(shape, seed, scale=1.0, dtype=torch.float32):
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32) * np.float32(scale)).to(dtype)


def spread(s, rows, cols, shape):
    s = np.repeat(np.repeat(s, rows, -2), cols, -1)
    return s[..., : shape[-2], : shape[-1]]


def e4m3_grid():
    """The non-negative E4M3 values in order."""
    v = [m * 2.0**-9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)]
    return np.array(v[:127])  # the last pattern is NaN


GRID = e4m3_grid()


def nearest_e4m3(v):
    """Nearest E4M3 value of a float64 array with |v| <= 448, ties to the even pattern."""
    a = np.abs(v)
    hi = np.searchsorted(GRID, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - GRID[lo], GRID[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.sign(v) * GRID[pick]


def block_max(x, rows, cols):
    m, k = x.shape
    p = np.zeros((blocks(m) * rows if rows > 1 else m, blocks(k) * cols))
    p[:m, :k] = np.abs(x)
    return p.reshape(p.shape[0] // rows, rows, p.shape[1] // cols, cols).max((1, 3))


def quantise_reference(x, rows):
    a = np.maximum(block_max(x, rows, 128), 2.0**-60)
    return nearest_e4m3(x * 448.0 / spread(a, rows, 128, x.shape)), a / 448.0


def random_f8(m, k, seed, ld=None, offset=0):
    """Random E4M3 values (device, rows `ld` apart from `offset`) and the same as float64."""
    r = np.random.default_rng(seed)
    v = GRID[r.integers(0, 127, (m, k))] * r.choice([-1.0, 1.0], (m, k))
    ld = ld or -(-k // 16) * 16
    buf = torch.zeros(offset + m * ld + 16, dtype=torch.uint8, device="cuda").view(F8)
    q = buf[offset : offset + m * ld].view(m, ld)[:, :k]
    q.copy_(torch.from_numpy(v).float().cuda().to(F8))
    return q, v


def random_scales(shape, seed):
    r = np.random.default_rng(seed)
    s = np.exp2(r.uniform(-12, 4, shape)).astype(np.float32)
    return torch.from_numpy(s).cuda(), s.astype(np.float64)


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------


def check_quantised(got, x, form):
    want = []
    if form == "tiles":
        want = [quantise_reference(x, 128)]
    else:
        want += [quantise_reference(x, 1)] if form in ("rows", "both") else []
        want += [quantise_reference(x.T, 1)] if form in ("columns", "both") else []
    assert len(got) == 2 * len(want)
    for (q, s), (gq, gs) in zip(want, zip(got[::2], got[1::2])):
        assert gq.dtype == F8 and gs.dtype == torch.float32
        assert gq.shape == q.shape and tuple(gs.shape) == s.shape
        np.testing.assert_array_equal(gs.cpu().numpy(), s.astype(np.float32))  # a correctly rounded division
        np.testing.assert_array_equal(gq.float().cpu().numpy(), q)


@pytest.mark.parametrize("form", ["rows", "columns", "both", "tiles"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 4096), (3, 100), (128, 128), (129, 127), (130, 391), (257, 1032)])
def test_quantise(rg, form, dtype, m, k):  # noqa: F811
    # 16-bit entries: the library's correctly rounded quotient cannot cross an E4M3 tie; fp32 entries are drawn on
    # a 16-bit grid here for the same reason
    x = normal((m, k), 1000 * m + k, 3.0, torch.bfloat16 if dtype == torch.float32 else dtype).to(dtype)
    check_quantised(rg.quantize_f8(x.cuda(), form), x.double().numpy(), form)


@pytest.mark.parametrize("m,k,dtype", [(601, 7100, torch.bfloat16), (4200, 1001, torch.float16)])
def test_quantise_many_row_blocks(rg, m, k, dtype):  # noqa: F811
    x = normal((m, k), m, 3.0, dtype)
    check_quantised(rg.quantize_f8(x.cuda(), "rows"), x.double().numpy(), "rows")


@pytest.mark.parametrize("form", ["rows", "columns", "both", "tiles"])
def test_quantise_strides_and_alignment(rg, form):  # noqa: F811
    base = normal((300, 701), 5, 1.0, torch.bfloat16).cuda()
    for x in (base[:, 1:], base[7:135, 3:259], base.t(), base[:, ::2], base[5:6, 9:]):
        check_quantised(rg.quantize_f8(x, form), x.double().cpu().numpy(), form)


@pytest.mark.parametrize("form", ["rows", "columns", "tiles"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantise_extreme_values(rg, form, dtype):  # noqa: F811
    """Blocks of zeros, of values below the smallest scale, next to the largest finite value, and E4M3 ties."""
    x = torch.zeros((256, 256), dtype=dtype)
    x[:, 128:] = normal((256, 128), 9, 2.0**-70, dtype)  # scaled as if their largest were 2^-60
    x[128:, :128] = normal((128, 128), 10, 1.0, dtype) * (torch.finfo(dtype).max / 8)
    x[130, 5] = torch.finfo(dtype).max
    x[128:, 128:] = (torch.arange(128 * 128).view(128, 128) % 255 - 127).to(dtype) * 0.5  # halves: ties
    x[128:, 128] = 448.0
    x[128, 128:] = 448.0
    check_quantised(rg.quantize_f8(x.cuda(), form), x.double().numpy(), form)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("form,rows", [("rows", 1), ("columns", 1), ("tiles", 128)])
def test_quantise_nonfinite_blocks(rg, bad, form, rows):  # noqa: F811
    x = normal((200, 300), 3)
    x[17, 140] = bad
    q, s = rg.quantize_f8(x.cuda(), form)
    v = q.double().cpu().numpy() * spread(s.double().cpu().numpy(), rows, 128, tuple(q.shape))
    xx = x.double().numpy().T if form == "columns" else x.double().numpy()
    i, j = (140, 17) if form == "columns" else (17, 140)
    hit = np.zeros(xx.shape, bool)
    hit[i // rows * rows : i // rows * rows + rows, j // 128 * 128 : j // 128 * 128 + 128] = True
    assert np.isnan(v[hit]).all() and np.isfinite(v[~hit]).all()


def test_quantise_empty(rg):  # noqa: F811
    for m, k in ((0, 5), (5, 0), (0, 0)):
        q, s, qt, st = rg.quantize_f8(torch.zeros((m, k), device="cuda"), "both")
        assert q.shape == (m, k) and s.shape == (m, blocks(k)) and qt.shape == (k, m) and st.shape == (k, blocks(m))


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------


def check_product(rg, m, n, k, transb, tile, out, seed=0, **kw):  # noqa: F811
    A, a = random_f8(m, k, seed + 1, **kw)
    B, b = random_f8(n, k, seed + 2, **kw) if transb else random_f8(k, n, seed + 2, **kw)
    SA, sa = random_scales((m, blocks(k)), seed + 3)
    nb = blocks(n) if tile else n
    SB, sb = random_scales((nb, blocks(k)) if transb else (blocks(k), nb), seed + 4)
    C = rg.scaled_gemm_f8(A, SA, B, SB, out_dtype=out, transb=transb)
    assert C.shape == (m, n) and C.dtype == out
    rows = 128 if tile else 1
    av = a * spread(sa, 1, 128, a.shape)
    bv = b * spread(sb, rows, 128, b.shape) if transb else (b.T * spread(sb.T, rows, 128, b.T.shape))
    ref, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    if out == torch.float16:  # beyond its range the result is inf
        ref = np.where(np.abs(ref) >= 65520.0, np.sign(ref) * np.inf, ref)
    got = C.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        bound = (144 + blocks(k)) * 2.0**-23 * mag + U[out] * np.abs(ref)
        if out == torch.float16:
            bound = bound + 2.0**-25  # half a subnormal step
            near = np.abs(np.abs(av @ bv.T) - 65520.0) <= (144 + blocks(k)) * 2.0**-23 * mag
        else:
            near = np.zeros(got.shape, bool)
        ok = (got == ref) | (np.abs(got - ref) <= bound) | near
    assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], ref[~ok][:5], bound[~ok][:5])
    return C


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 300, 2000), (7, 33, 65), (8, 1000, 1024), (17, 129, 257), (33, 4096, 512),
          (64, 64, 4096), (128, 128, 128), (130, 260, 1000), (255, 257, 384), (300, 512, 127), (1000, 776, 520)]


@pytest.mark.parametrize("transb", [True, False])
@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(rg, m, n, k, transb, tile):  # noqa: F811
    check_product(rg, m, n, k, transb, tile, torch.float32)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k,transb", [(1, 515, 640, True), (24, 256, 300, True), (200, 391, 512, False),
                                          (513, 640, 1100, True)])
def test_product_16_bit_results(rg, m, n, k, transb, out):  # noqa: F811
    check_product(rg, m, n, k, transb, True, out, seed=50)


@pytest.mark.parametrize("m,n,k,transb,tile", [(2100, 2300, 640, True, True), (2048, 2304, 1025, False, True),
                                               (2050, 2177, 333, True, False), (1, 70000, 128, True, True),
                                               (70000, 16, 130, False, False)])
def test_product_many_tiles(rg, m, n, k, transb, tile):  # noqa: F811
    check_product(rg, m, n, k, transb, tile, torch.float32, seed=70)


@pytest.mark.parametrize("transb,tile", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("m,n,k,out", [(1, 1, 1, torch.float32), (130, 260, 1000, torch.float32),
                                       (257, 513, 200, torch.bfloat16), (520, 392, 2100, torch.float32),
                                       (300, 200, 640, torch.float16)])
def test_product_kernels(rg, variant, m, n, k, out, transb, tile):  # noqa: F811
    """Both tensor-core kernels, whatever the shape would choose."""
    check_product(rg, m, n, k, transb, tile, out, seed=90)


def test_product_long_k(rg):  # noqa: F811
    check_product(rg, 40, 50, 70001, True, False, torch.float32, seed=80)
    check_product(rg, 3, 200, 70001, True, True, torch.float32, seed=81)


def test_product_row_strides_and_offsets(rg):  # noqa: F811
    check_product(rg, 70, 90, 200, True, True, torch.float32, ld=304)  # padded rows
    check_product(rg, 70, 208, 300, False, True, torch.float32, ld=320, offset=48)
    check_product(rg, 70, 90, 201, True, True, torch.float32, ld=201)  # rows off 16-byte boundaries: copied
    check_product(rg, 5, 90, 201, True, True, torch.float32, ld=208, offset=3)


def test_product_nonfinite_scales_stay_in_their_rows(rg):  # noqa: F811
    A, a = random_f8(40, 300, 1)
    B, b = random_f8(150, 300, 2)
    SA, _ = random_scales((40, 3), 3)
    SB, _ = random_scales((2, 3), 4)
    SA[7, 1] = float("nan")
    SB[1, 2] = float("inf")
    C = rg.scaled_gemm_f8(A, SA, B, SB, out_dtype=torch.float32, transb=True).cpu().numpy()
    assert np.isnan(C[7]).all()
    rest = np.delete(C, 7, 0)
    assert np.isfinite(rest[:, :128]).all() and not np.isfinite(rest[:, 128:]).any()


def test_product_of_nan_values(rg):  # noqa: F811
    A, _ = random_f8(20, 260, 1)
    B, _ = random_f8(140, 260, 2)
    A.view(torch.uint8)[3, 259] = 0x7F
    B.view(torch.uint8)[130, 0] = 0xFF
    for m in (20, 4):
        C = rg.scaled_gemm_f8(A[:m], torch.ones((m, 3), device="cuda"), B, torch.ones((2, 3), device="cuda"),
                              out_dtype=torch.float32, transb=True).cpu().numpy()
        want = np.zeros((m, 140), bool)
        want[3] = True
        want[:, 130] = True
        assert (np.isnan(C) == want).all()


def test_product_empty(rg):  # noqa: F811
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    e = lambda *s: torch.zeros(s, device="cuda").to(F8)  # noqa: E731
    C = rg.scaled_gemm_f8(e(3, 0), one(3, 0), e(5, 0), one(1, 0), transb=True)
    assert C.shape == (3, 5) and (C == 0).all()
    assert rg.scaled_gemm_f8(e(0, 7), one(0, 1), e(5, 7), one(1, 1), transb=True).shape == (0, 5)
    assert rg.scaled_gemm_f8(e(3, 7), one(3, 1), e(7, 0), one(1, 0)).shape == (3, 0)


def test_product_out_and_repeats(rg):  # noqa: F811
    A, _ = random_f8(130, 2000, 1)
    B, _ = random_f8(260, 2000, 2)
    SA, _ = random_scales((130, 16), 3)
    SB, _ = random_scales((260, 16), 4)
    out = torch.empty((130, 260), dtype=torch.float32, device="cuda")
    first = rg.scaled_gemm_f8(A, SA, B, SB, out_dtype=torch.float32, transb=True)
    assert rg.scaled_gemm_f8(A, SA, B, SB, out_dtype=torch.float32, transb=True, out=out) is out
    assert torch.equal(out, first)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        other = rg.scaled_gemm_f8(A, SA, B, SB, out_dtype=torch.float32, transb=True, sync=False)
    s.synchronize()
    assert torch.equal(other, first)


def test_product_timeout_is_reported(rg, variant):  # noqa: F811
    """A product whose tensor-core stage never reports its first block ends with a time-out, and the next is sound."""
    lib = rg.library()
    A, _ = random_f8(512, 512, 1)
    B, _ = random_f8(512, 512, 2)
    SA, _ = random_scales((512, 4), 3)
    SB, _ = random_scales((4, 4), 4)
    good = rg.scaled_gemm_f8(A, SA, B, SB, transb=True)
    old = lib.rg_set_wait_limit_ns(50_000_000)
    try:
        lib.rg_inject_fault(1)
        with pytest.raises(rg.ResGemmError) as err:
            rg.scaled_gemm_f8(A, SA, B, SB, transb=True)
        assert err.value.code == rg.RG_ERR_TIMEOUT
    finally:
        lib.rg_inject_fault(0)
        lib.rg_set_wait_limit_ns(old)
    assert torch.equal(rg.scaled_gemm_f8(A, SA, B, SB, transb=True), good)


# ---------------------------------------------------------------------------
# linear layer
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("m,n,k,dtype", [(1, 130, 200, torch.bfloat16), (200, 136, 264, torch.bfloat16),
                                         (131, 257, 129, torch.float16)])
def test_linear_gradients(rg, m, n, k, dtype):  # noqa: F811
    x, w = normal((m, k), 1, 1.0, dtype), normal((n, k), 2, k**-0.5, torch.bfloat16).float()
    dy = normal((m, n), 3, 2.0**-4, dtype)
    Y, saved = rg.linear_f8(x.cuda(), w.cuda())
    dX, dW = rg.linear_f8_backward(dy.cuda(), saved)
    assert Y.dtype == dX.dtype == dtype and dW.dtype == torch.float32
    xd, wd, dd = x.double().numpy(), w.double().numpy(), dy.double().numpy()

    def value(z, rows):
        q, s = quantise_reference(z, rows)
        return q * spread(s, rows, 128, z.shape)

    qw = value(wd, 128)
    for got, a, b in ((Y, value(xd, 1), qw.T), (dX, value(dd, 1), qw), (dW, value(dd.T, 1), value(xd.T, 1).T)):
        ref, mag = a @ b, np.abs(a) @ np.abs(b)
        # scales are fp32: one rounding (2^-24) on each side more than in a product of given scales
        bound = (146 + blocks(a.shape[1])) * 2.0**-23 * mag + U[got.dtype] * np.abs(ref) + 2.0**-24
        assert (np.abs(got.double().cpu().numpy() - ref) <= bound).all()

    # against differences of the unquantised layer, which is linear in x and in w: a quantised entry is within
    # 2^-4 of its own or 2^-10 of its scale of the entry, so a product of two is within e1|b| + |a|e2 + e1 e2
    def off(z, rows):
        s = spread(np.maximum(block_max(z, rows, 128), 2.0**-60) / 448.0, rows, 128, z.shape)
        return np.maximum(np.abs(z) * 2.0**-4, s * 2.0**-10)

    v = np.random.default_rng(4).standard_normal((m, k))
    loss = lambda xx, ww: (dd * (xx @ ww.T)).sum()  # noqa: E731
    slope = (loss(xd + v / 2, wd) - loss(xd - v / 2, wd))
    ed, ew = off(dd, 1), off(wd, 128)
    tol = (np.abs(v) * (ed @ np.abs(wd) + np.abs(dd) @ ew + ed @ ew)).sum()
    tol += (np.abs(v) * (U[dtype] * 2 * np.abs(dd) @ np.abs(wd) + 2.0**-24)).sum()
    assert abs((dX.double().cpu().numpy() * v).sum() - slope) <= tol
    v = np.random.default_rng(5).standard_normal((n, k))
    slope = loss(xd, wd + v / 2) - loss(xd, wd - v / 2)
    ed, ex = off(dd.T, 1), off(xd.T, 1).T
    tol = (np.abs(v) * (ed @ np.abs(xd) + np.abs(dd.T) @ ex + ed @ ex)).sum()
    tol += (np.abs(v) * (2.0**-14 * np.abs(dd.T) @ np.abs(xd))).sum()
    assert abs((dW.double().cpu().numpy() * v).sum() - slope) <= tol


def test_linear_is_its_parts(rg):  # noqa: F811
    """The layer's calls give what quantisation and products give one after the other, strided inputs included."""
    x = normal((300, 270), 1, 1.0, torch.bfloat16).cuda()[:, 5:261]
    w = normal((256, 200), 2, 0.1).cuda().t()  # [200, 256], columns contiguous
    dy = normal((300, 400), 3, 0.01, torch.bfloat16).cuda()[:, ::2]
    Y, saved = rg.linear_f8(x, w)
    dX, dW = rg.linear_f8_backward(dy, saved, dw_dtype=torch.bfloat16)
    qx, sx, qxt, sxt = rg.quantize_f8(x, "both")
    qw, sw = rg.quantize_f8(w, "tiles")
    qd, sd, qdt, sdt = rg.quantize_f8(dy, "both")
    assert torch.equal(Y, rg.scaled_gemm_f8(qx, sx, qw, sw, transb=True))
    assert torch.equal(dX, rg.scaled_gemm_f8(qd, sd, qw, sw))
    assert torch.equal(dW, rg.scaled_gemm_f8(qdt, sdt, qxt, sxt, transb=True))


@pytest.mark.parametrize("dtype,dw", [(torch.bfloat16, torch.float32), (torch.float16, torch.float16),
                                      (torch.float32, torch.bfloat16)])
def test_linear_ordinary_call_is_its_parts(rg, dtype, dw):  # noqa: F811
    """Contiguous tensors, the second call on a warm workspace: the native call path."""
    x, w, dy = normal((70, 200), 1, 1.0, dtype).cuda(), normal((96, 200), 2).cuda(), normal((70, 96), 3, 0.1, dtype).cuda()
    qx, sx, qxt, sxt = rg.quantize_f8(x, "both")
    qw, sw = rg.quantize_f8(w, "tiles")
    qd, sd, qdt, sdt = rg.quantize_f8(dy, "both")
    for _ in range(2):
        Y, saved = rg.linear_f8(x, w)
        dX, dW = rg.linear_f8_backward(dy, saved, dw_dtype=dw)
        assert Y.dtype == dX.dtype == dtype and dW.dtype == dw
        assert torch.equal(Y, rg.scaled_gemm_f8(qx, sx, qw, sw, transb=True, out_dtype=dtype))
        assert torch.equal(dX, rg.scaled_gemm_f8(qd, sd, qw, sw, out_dtype=dtype))
        assert torch.equal(dW, rg.scaled_gemm_f8(qdt, sdt, qxt, sxt, transb=True, out_dtype=dw))


def test_linear_saved_buffer_is_checked(rg):  # noqa: F811
    """A buffer shorter than the forward pass made, and a gradient of another shape or type, are refused."""
    x, w = normal((70, 200), 1).cuda(), normal((96, 200), 2).cuda()
    Y, (kept, M, N, K) = rg.linear_f8(x, w)
    with pytest.raises(rg.ResGemmError) as err:
        rg.linear_f8_backward(Y, (kept[:-256], M, N, K))
    assert err.value.code == rg.RG_ERR_WORKSPACE
    for dy, dw in ((Y[:, :-1], torch.float32), (Y[:-1], torch.float32), (Y.double(), torch.float32),
                   (Y, torch.float64)):
        with pytest.raises(ValueError):
            rg.linear_f8_backward(dy, (kept, M, N, K), dw_dtype=dw)


def test_linear_empty(rg):  # noqa: F811
    x, w = torch.zeros((0, 40), device="cuda"), torch.ones((30, 40), device="cuda")
    Y, saved = rg.linear_f8(x, w)
    dX, dW = rg.linear_f8_backward(Y, saved)
    assert Y.shape == (0, 30) and dX.shape == (0, 40) and dW.shape == (30, 40) and (dW == 0).all()


def test_linear_backward_reports_its_first_product(rg):  # noqa: F811
    """A time-out in the input gradient's product is not hidden by the weight gradient's that follows it."""
    lib = rg.library()
    x, w = normal((300, 256), 1).cuda(), normal((256, 256), 2).cuda()
    Y, saved = rg.linear_f8(x, w)
    old = lib.rg_set_wait_limit_ns(50_000_000)
    try:
        lib.rg_inject_fault(1)
        with pytest.raises(rg.ResGemmError) as err:
            rg.linear_f8_backward(Y, saved)
        assert err.value.code == rg.RG_ERR_TIMEOUT
    finally:
        lib.rg_inject_fault(0)
        lib.rg_set_wait_limit_ns(old)
    rg.linear_f8_backward(Y, saved)


# ---------------------------------------------------------------------------
# mixture of experts
# ---------------------------------------------------------------------------


def moe_inputs(t, h, i, e, dtype, seed, x_scale=1.0):
    x = normal((t, h), seed, x_scale, dtype)
    wr = normal((e, h), seed + 1, h**-0.5, dtype)
    r = np.random.default_rng(seed + 2)

    def weights(n, k):
        q = GRID[r.integers(0, 127, (e, n, k))] * r.choice([-1.0, 1.0], (e, n, k))
        s = np.exp2(r.uniform(-1, 1, (e, blocks(n), blocks(k)))).astype(np.float32)
        s *= np.float32(k**-0.5 / 150.0)
        return torch.from_numpy(q).float().to(F8), torch.from_numpy(s)

    return (x, wr) + weights(2 * i, h) + weights(h, i)


def moe_reference(x, wr, w13, s13, w2, s2, top_k, renorm):
    """(y, bound on a float32 result before its last rounding) in 64 bits; token by token, expert by expert."""
    x, wr = x.double().numpy(), wr.double().numpy()
    w13 = w13.double().numpy() * spread(s13.double().numpy(), 128, 128, tuple(w13.shape))
    w2 = w2.double().numpy() * spread(s2.double().numpy(), 128, 128, tuple(w2.shape))
    t, h = x.shape
    i = w2.shape[2]
    u = 2.0**-23
    c1, c2 = 8 * 17 + blocks(h) + 12, 8 * 17 + blocks(i) + 12  # units per sum of |products|, as for a product
    y, err = np.zeros((t, h)), np.zeros((t, h))
    for r in range(t):
        logits = wr @ x[r]
        dl = (h * 2.0**-24 * (np.abs(wr) @ np.abs(x[r]))).max()
        order = np.argsort(-logits, kind="stable")
        if len(order) > top_k:  # the choice must not hang on rounding
            assert logits[order[top_k - 1]] - logits[order[top_k]] > 2 * dl or \
                logits[order[top_k - 1]] == logits[order[top_k]]
        p = np.exp(logits - logits.max())
        p /= p.sum()
        sel = order[:top_k]
        g = p[sel] / (p[sel].sum() if renorm else 1.0)
        eg = 4 * dl + 64 * u  # relative: numerator, denominator, exp, sums, division
        for e, w in zip(sel, g):
            a, b = w13[e, :i] @ x[r], w13[e, i:] @ x[r]
            ax = np.abs(x[r]) + 2.0**-40 * np.abs(x[r]).max()
            ea, eb = c1 * u * (np.abs(w13[e, :i]) @ ax), c1 * u * (np.abs(w13[e, i:]) @ ax)
            silu = a / (1 + np.exp(-a))
            hh = silu * b
            eh = 1.1 * ea * (np.abs(b) + eb) + np.abs(silu) * eb + 8 * u * np.abs(hh)
            eh = eh + 2.0**-12 * (np.abs(hh) + eh) + 2.0**-27 * (np.abs(hh) + eh).max()
            o, mag = w2[e] @ hh, np.abs(w2[e]) @ (np.abs(hh) + eh)
            eo = np.abs(w2[e]) @ eh + c2 * u * mag
            y[r] += w * o
            err[r] += w * (eo + (eg + (top_k + 2) * u) * (np.abs(o) + eo))
    return y, err


def check_moe(rg, args, top_k, renorm):  # noqa: F811
    y, err = moe_reference(*args, top_k, renorm)
    Y = rg.moe_layer_f8(*(a.cuda() for a in args), top_k, renorm=renorm)
    assert Y.dtype == args[0].dtype
    bound = err + U[Y.dtype] * (np.abs(y) + err) + 2.0**-25
    bad = ~(np.abs(Y.double().cpu().numpy() - y) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], Y.double().cpu().numpy()[bad][:4], y[bad][:4], bound[bad][:4])
    return Y


@pytest.mark.parametrize("t,h,i,e,top_k,renorm", [
    (1, 16, 16, 1, 1, True), (1, 256, 128, 8, 2, True), (1, 528, 272, 64, 8, False), (2, 272, 80, 5, 5, False),
    (5, 400, 144, 33, 4, True), (9, 1040, 208, 3, 1, True), (17, 256, 256, 2, 2, False), (33, 160, 112, 4, 3, True),
    (64, 144, 176, 1, 1, True), (64, 512, 128, 100, 6, True), (64, 192, 64, 17, 16, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_moe(rg, t, h, i, e, top_k, renorm, dtype):  # noqa: F811
    check_moe(rg, moe_inputs(t, h, i, e, dtype, 31 * t + h), top_k, renorm)


def test_moe_many_experts(rg):  # noqa: F811
    check_moe(rg, moe_inputs(3, 128, 32, 512, torch.bfloat16, 3), 16, True)


def test_moe_equal_logits_take_the_lowest_experts(rg):  # noqa: F811
    args = list(moe_inputs(4, 256, 64, 40, torch.bfloat16, 8))
    args[1] = torch.zeros_like(args[1])
    args[1][::2] = -0.0  # zeros of both signs tie
    check_moe(rg, tuple(args), 6, True)
    args[1][5] = args[1][37] = args[0][0] * 0.01  # two equal largest for token 0
    y, _ = moe_reference(*args, 1, True)
    Y = rg.moe_layer_f8(*(a.cuda() for a in args), 1)
    np.testing.assert_allclose(Y[0].double().cpu().numpy(), y[0], atol=0.02 * np.abs(y[0]).max())


@pytest.mark.parametrize("scale", [2.0**-60, 2.0**50])
def test_moe_magnitudes(rg, scale):  # noqa: F811
    """Activations far outside fp16's range: the scaled fp16 operands must neither overflow nor vanish."""
    args = list(moe_inputs(5, 256, 128, 6, torch.bfloat16, 12, scale))
    args[1] = (args[1].float() / scale).to(torch.bfloat16)  # logits of ordinary size
    if scale > 1:  # h grows with the square of x: keep the gate ordinary by small gate weights
        args[3] = args[3].clone()
        args[3] *= 2.0**-40
    check_moe(rg, tuple(args), 2, True)


def test_moe_nonfinite_tokens_stay_in_their_rows(rg):  # noqa: F811
    args = list(moe_inputs(6, 256, 64, 8, torch.bfloat16, 21))
    good = rg.moe_layer_f8(*(a.cuda() for a in args), 2)
    args[0][1, 7] = float("nan")
    args[0][4, 200] = float("inf")
    Y = rg.moe_layer_f8(*(a.cuda() for a in args), 2)
    assert torch.isnan(Y[[1, 4]]).all()
    assert torch.equal(Y[[0, 2, 3, 5]], good[[0, 2, 3, 5]])


def test_moe_a_token_alone_and_in_a_batch(rg):  # noqa: F811
    """Equal calls give equal bits, and a token's result is the same whatever tokens come with it when its experts
    see at most eight tokens."""
    args = [a.cuda() for a in moe_inputs(8, 512, 128, 16, torch.bfloat16, 40)]
    Y = rg.moe_layer_f8(*args, 4)
    for _ in range(3):
        assert torch.equal(rg.moe_layer_f8(*args, 4), Y)
    for t in range(8):
        assert torch.equal(rg.moe_layer_f8(args[0][t : t + 1], *args[1:], 4)[0], Y[t])


def test_moe_empty_and_streams(rg):  # noqa: F811
    args = [a.cuda() for a in moe_inputs(3, 256, 64, 8, torch.bfloat16, 50)]
    assert rg.moe_layer_f8(args[0][:0], *args[1:], 2).shape == (0, 256)
    want = rg.moe_layer_f8(*args, 2)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        got = rg.moe_layer_f8(*args, 2, sync=False)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    off = torch.zeros(3 * 256 + 1, dtype=torch.bfloat16, device="cuda")
    off[1:] = args[0].reshape(-1)  # tokens off a 16-byte boundary
    assert rg.moe_layer_f8(off[1:].view(3, 256), *args[1:], 2, out=out) is out
    assert torch.equal(out, want)


def test_example_trains_and_decodes(rg):  # noqa: F811
    """The example's layer learns (its loss falls to the quantisation's noise) and its decoding is finite."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import f8_layers

    losses, w = f8_layers.train()
    # the target's outputs have variance 1; E4M3 keeps every factor of a product within 2^-4
    assert losses[0] > 0.5 and losses[-1] < (2 * 2.0**-4) ** 2 * losses[0]
    y, z = f8_layers.decode(w)
    assert torch.isfinite(y).all() and torch.isfinite(z).all() and float(z.float().abs().max()) > 0


def test_graph_capture(rg):  # noqa: F811
    """Quantisation, product and expert layer replay from a CUDA graph on new inputs."""
    x = normal((4, 256), 1, 1.0, torch.bfloat16).cuda()
    w = normal((384, 256), 2, 0.1).cuda()
    args = [a.cuda() for a in moe_inputs(4, 256, 64, 8, torch.bfloat16, 60)]
    qw, sw = rg.quantize_f8(w, "tiles")

    def step():
        q, s = rg.quantize_f8(x, "rows", sync=False)
        return (rg.scaled_gemm_f8(q, s, qw, sw, transb=True, sync=False),
                rg.moe_layer_f8(x, *args[1:], 2, sync=False))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    x.copy_(normal((4, 256), 77, 2.0, torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, step()):
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    assert math.isfinite(float(outs[0].float().abs().sum()))
