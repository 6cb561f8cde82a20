"""8-bit products by group of rows against plain 64-bit implementations.

Bounds: those of the other 8-bit products (test_gpu_f8.py): |error| <= (144 + KB) 2^-23 sum |a b| + u |c|, KB blocks
of 128 along the contraction; two more units where scales come from the quantisation.
"""
import numpy as np
import pytest
import torch

from gpu_util import rg, variant  # noqa: F401
from test_gpu_f8 import F8, U, block_max, blocks, normal, quantise_reference, random_f8, random_scales, spread

pytestmark = pytest.mark.gpu

COUNTS = {
    "one row": [1],
    "one group": [300],
    "even": [128, 256, 128],
    "ragged": [1, 0, 127, 129, 0, 0, 300, 5],
    "first and last empty": [0, 40, 2, 0],
    "no rows": [0, 0, 0],
    "single rows": [0, 1, 0, 0, 1, 1, 0, 1],
    "large": [700, 3, 513, 256],
}


def offsets_of(counts, dtype=torch.int32):
    return torch.tensor([0, *np.cumsum(counts)], dtype=dtype, device="cuda")


def starts(counts):
    """First block of each group along the rows."""
    off = np.concatenate([[0], np.cumsum(counts)])
    return [int(off[g]) // 128 + g for g in range(len(counts))]


def stack_f8(e, m, k, seed):
    """Random E4M3 matrices, rows on 16-byte boundaries, without gaps between them."""
    q, v = random_f8(e * m, k, seed)
    return q.as_strided((e, m, k), (m * q.stride(0), q.stride(0), 1)), v.reshape(e, m, k)


def close(C, ref, mag, kb, extra=0):
    got, u = C.double().cpu().numpy(), U[C.dtype]
    bound = (144 + extra + kb) * 2.0**-23 * mag + u * np.abs(ref) + (2.0**-25 if C.dtype == torch.float16 else 0)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], bound[bad][:5])


def check_rows(rg, counts, n, k, transb, out, pad=0, seed=0, dtype=torch.int32):  # noqa: F811
    e, t = len(counts), sum(counts) + pad
    A, a = random_f8(t, k, seed + 1)
    B, b = stack_f8(e, n, k, seed + 2) if transb else stack_f8(e, k, n, seed + 2)
    SA, sa = random_scales((t, blocks(k)), seed + 3)
    SB, sb = random_scales((e, blocks(n), blocks(k)) if transb else (e, blocks(k), blocks(n)), seed + 4)
    if out == torch.float16:  # within its range
        SA, sa = SA * 2.0**-6, sa * 2.0**-6
        SB, sb = SB * 2.0**-12, sb * 2.0**-12
    C = rg.grouped_gemm_f8(A, SA, B, SB, offsets_of(counts, dtype), out_dtype=out, transb=transb)
    assert C.shape == (t, n) and C.dtype == out
    av = a * spread(sa, 1, 128, a.shape)
    ref, mag = np.zeros((t, n)), np.zeros((t, n))
    at = 0
    for g, c in enumerate(counts):
        bv = b[g] * spread(sb[g], 128, 128, b[g].shape)
        bv = bv.T if transb else bv
        ref[at : at + c], mag[at : at + c] = av[at : at + c] @ bv, np.abs(av[at : at + c]) @ np.abs(bv)
        at += c
    close(C, ref, mag, blocks(k))
    return A, SA, B, SB, C


@pytest.mark.parametrize("transb", [True, False])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(1, 1), (130, 260), (392, 1100)])
def test_rows(rg, variant, counts, n, k, transb):  # noqa: F811
    check_rows(rg, COUNTS[counts], n, k, transb, torch.float32, seed=n)


@pytest.mark.parametrize("transb", [True, False])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,k,pad", [(257, 129, 0), (512, 384, 150), (80, 2056, 1)])
def test_rows_16_bit_results(rg, variant, n, k, pad, out, transb):  # noqa: F811
    check_rows(rg, COUNTS["ragged"], n, k, transb, out, pad, seed=20, dtype=torch.int64)


@pytest.mark.parametrize("transb", [True, False])
@pytest.mark.parametrize("per", [4, 100, 200])
def test_rows_of_many_groups(rg, per, transb):  # noqa: F811
    """More units than SMs, by the kernel that the average chooses."""
    counts = np.random.default_rng(per).integers(0, 2 * per, 40).tolist()
    check_rows(rg, counts, 1160, 650, transb, torch.bfloat16, pad=per, seed=per)


def test_most_groups(rg, variant):  # noqa: F811
    counts = np.random.default_rng(1).integers(0, 3, 512).tolist()
    check_rows(rg, counts, 140, 130, True, torch.float32, pad=3, seed=5)


@pytest.mark.parametrize("k", [1, 300])
def test_rows_are_their_groups_product(rg, variant, k):  # noqa: F811
    """Checked in 64 bits, and on the CTA-pair kernel the same sums as each group's own product, to the bit."""
    counts = [3, 0, 200, 61]
    A, SA, B, SB, C = check_rows(rg, counts, 300, k, True, torch.float32, seed=3)
    at = 0
    for g, c in enumerate(counts):
        if c and variant == 2:
            one = rg.scaled_gemm_f8(A[at : at + c], SA[at : at + c], B[g], SB[g], out_dtype=torch.float32, transb=True)
            assert torch.equal(C[at : at + c], one)
        at += c


def test_rows_behind_the_last_group(rg, variant):  # noqa: F811
    """Zeros in a new result; left as they were in a given one."""
    A, SA, B, SB, C = check_rows(rg, [5, 200, 0], 140, 200, True, torch.float32, pad=170)
    assert (C[205:] == 0).all()
    out = torch.full_like(C, 7.0)
    assert rg.grouped_gemm_f8(A, SA, B, SB, offsets_of([5, 200, 0]), torch.float32, True, out=out) is out
    assert torch.equal(out[:205], C[:205]) and (out[205:] == 7).all()


def test_rows_strides_and_alignment(rg, variant):  # noqa: F811
    counts = [3, 40, 70]
    A, SA, B, SB, C = check_rows(rg, counts, 100, 200, True, torch.float32, seed=9)
    off = offsets_of(counts)
    plain = B.contiguous()  # rows of 200 bytes: copied
    spaced = torch.zeros((6, 100, 208), device="cuda").to(F8)[::2, :, :200]  # gaps between the matrices: copied
    spaced.copy_(B)
    wide = torch.zeros((113, 320), device="cuda").to(F8)[:, 16:216]
    wide.copy_(A)
    for a, b, o in ((A, plain, off), (A, spaced, off), (wide, B, off), (A[:, :], B, off.repeat_interleave(2)[::2])):
        assert torch.equal(rg.grouped_gemm_f8(a, SA, b, SB, o, torch.float32, True), C)
    odd = torch.empty(113 * 100 + 1, device="cuda")[1:].view(113, 100)  # results off 16-byte boundaries
    assert torch.equal(rg.grouped_gemm_f8(A, SA, B, SB, off, torch.float32, True, out=odd), C)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [256, 252, 250, 249])
def test_products_on_every_boundary(rg, variant, n, dtype):  # noqa: F811
    """By rows and summed over them, results 0, 1, 2, 4 entries off 16-byte boundaries: bits as on them, and rows behind
    the last group and memory beside the result left alone."""
    counts, m = [3, 130, 0, 300], 136
    off = offsets_of(counts)
    T, E = sum(counts) + 5, len(counts)
    A, SA, B, SB, C = check_rows(rg, counts, 256, 384, True, dtype, seed=9)
    XA, XS = rg.quantize_f8(torch.randn((T, m), device="cuda"), "columns", offsets=off)
    Y = torch.randn((T, 256), device="cuda")
    YB, YS = rg.quantize_f8(Y, "columns", offsets=off)
    want = rg.grouped_wgrad_f8(XA, XS, YB, YS, off, out_dtype=dtype)
    B, SB = B[:, :n].contiguous(), SB[:, : -(-n // 128)].contiguous()
    YB, YS = YB[:n], YS[:n]
    rows = C.shape[0]
    for shift in (0, 1, 2, 4):
        buf = torch.full((rows * n + 16,), 7.0, dtype=dtype, device="cuda")
        out = buf[shift : shift + rows * n].view(rows, n)
        rg.grouped_gemm_f8(A, SA, B, SB, off, dtype, True, out=out)
        assert torch.equal(out[: sum(counts)], C[: sum(counts), :n])
        assert (out[sum(counts) :] == 7).all() and (buf[:shift] == 7).all() and (buf[shift + rows * n :] == 7).all()
        buf = torch.full((E * m * n + 16,), 7.0, dtype=dtype, device="cuda")
        out = buf[shift : shift + E * m * n].view(E, m, n)
        rg.grouped_wgrad_f8(XA, XS, YB, YS, off, out=out, out_dtype=dtype)
        assert torch.equal(out, want[:, :, :n])
        assert (buf[:shift] == 7).all() and (buf[shift + E * m * n :] == 7).all()


@pytest.mark.parametrize("bad", [[1, 3, 9], [0, 5, 4], [0, 3, 11], [0, -1, 9], [0, 2**40, 9], [0, 3, 2**31 + 3],
                                 [-5, 0, 9]])
def test_bad_offsets_are_reported(rg, variant, bad):  # noqa: F811
    """Offsets that do not start at 0, fall or leave the rows: an error, and no entry of C is written."""
    A, _ = random_f8(10, 64, 1)
    B, _ = stack_f8(2, 32, 64, 2)
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    out = torch.full((10, 32), 7.0, device="cuda")
    off = torch.tensor(bad, device="cuda")
    with pytest.raises(rg.ResGemmError) as err:
        rg.grouped_gemm_f8(A, one(10, 1), B, one(2, 1, 1), off, torch.float32, True, out=out)
    assert err.value.code == rg.RG_ERR_ARG and (out == 7).all()
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    rg.grouped_gemm_f8(A, one(10, 1), B, one(2, 1, 1), off, torch.float32, True, sync=False, out=out, ws=ws)
    assert rg.status(ws) == rg.RG_ERR_ARG and (out == 7).all()
    rg.grouped_gemm_f8(A, one(10, 1), B, one(2, 1, 1), offsets_of([4, 6]), torch.float32, True, ws=ws)
    assert rg.status(ws) == rg.RG_OK


def test_nan_stays_in_its_rows(rg, variant):  # noqa: F811
    """A NaN in one group's rows or weights, or in rows behind the last group, reaches nothing else."""
    counts = [10, 0, 30]
    A, _ = random_f8(60, 200, 1)
    B, _ = stack_f8(3, 40, 200, 2)
    SA, _ = random_scales((60, 2), 3)
    SB, _ = random_scales((3, 1, 2), 4)
    A.view(torch.uint8)[4, 199] = 0x7F
    A.view(torch.uint8)[50] = 0x7F
    B.view(torch.uint8)[1] = 0xFF  # the group without rows
    B.view(torch.uint8)[2, 7, 0] = 0x7F
    C = rg.grouped_gemm_f8(A, SA, B, SB, offsets_of(counts), torch.float32, True)
    want = torch.zeros((60, 40), dtype=torch.bool, device="cuda")
    want[4] = True
    want[10:40, 7] = True
    assert torch.equal(torch.isnan(C), want) and (C[40:] == 0).all()
    # the contraction over ragged rows of the weights: the next matrix's values are beyond K, not part of it
    Bt, bt = stack_f8(2, 130, 40, 5)
    Bt.view(torch.uint8)[1] = 0x7F
    At, _ = random_f8(6, 130, 6)
    C = rg.grouped_gemm_f8(At, torch.ones((6, 2), device="cuda"), Bt, torch.ones((2, 2, 1), device="cuda"),
                           offsets_of([6, 0]), torch.float32)
    assert torch.isfinite(C).all()


# ---------------------------------------------------------------------------
# blocks along the rows, and sums over them
# ---------------------------------------------------------------------------


def grouped_reference(x, counts, pad):
    """(Q, S) of x's columns in blocks of one group each."""
    nb = (sum(counts) + pad) // 128 + len(counts)
    q, s = np.zeros((x.shape[1], 128 * nb)), np.full((x.shape[1], nb), 2.0**-60 / 448.0)
    at = 0
    for g0, c in zip(starts(counts), counts):
        if c:
            gq, gs = quantise_reference(x[at : at + c].T, 1)
            q[:, 128 * g0 : 128 * g0 + c], s[:, g0 : g0 + blocks(c)] = gq, gs
        at += c
    return q, s.astype(np.float32)


@pytest.mark.parametrize("form", ["columns", "both"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("counts,pad,k", [("one row", 0, 1), ("ragged", 0, 130), ("ragged", 300, 257), ("even", 1, 64),
                                          ("no rows", 0, 20), ("no rows", 129, 20), ("single rows", 127, 129),
                                          ("large", 40, 300), ("one group", 84, 16)])
def test_quantise_groups(rg, form, dtype, counts, pad, k):  # noqa: F811
    counts = COUNTS[counts]
    t = sum(counts) + pad
    x = normal((t, k), 7 * t + k, 3.0, torch.bfloat16 if dtype == torch.float32 else dtype).to(dtype)
    got = rg.quantize_f8(x.cuda(), form, offsets=offsets_of(counts, torch.int64 if k == 130 else torch.int32))
    q, s = grouped_reference(x.double().numpy(), counts, pad)
    np.testing.assert_array_equal(got[-2].float().cpu().numpy(), q)
    np.testing.assert_array_equal(got[-1].cpu().numpy(), s)
    if form == "both":
        for a, b in zip(got[:2], rg.quantize_f8(x.cuda(), "rows")):
            assert torch.equal(a.float(), b.float())


def test_quantise_groups_of_bad_offsets_stays_in_bounds(rg):  # noqa: F811
    """Whatever the offsets are, rows and places outside the matrices are neither read nor written."""
    guard = torch.full((3, 300, 40), 7.0, device="cuda", dtype=torch.bfloat16)
    x = guard[1]
    for bad in ([5, 3, 1], [0, -7, 300], [0, 2**40, 2**50], [400, 500, 600], [-(2**62), 2**62, 5], [300, 300, 300]):
        q, s, qt, st = rg.quantize_f8(x, "both", offsets=torch.tensor(bad, device="cuda"))
        assert qt.shape == (40, 128 * 4) and (guard == 7).all()


@pytest.mark.parametrize("e,n,k", [(1, 1, 1), (3, 130, 260), (5, 128, 64), (2, 257, 391), (512, 3, 20)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantise_stack(rg, e, n, k, dtype):  # noqa: F811
    w = normal((e, n, k), 3, 0.1, torch.bfloat16).to(dtype).cuda()
    q, s = rg.quantize_f8(w, "tiles")
    assert q.shape == (e, n, k) and s.shape == (e, blocks(n), blocks(k))
    for g in range(e):
        for a, b in zip((q[g], s[g]), rg.quantize_f8(w[g], "tiles")):
            assert torch.equal(a.float(), b.float())
    gaps = torch.zeros((2 * e, n, k), dtype=dtype, device="cuda")[::2]
    gaps.copy_(w)
    turned = w.transpose(1, 2).contiguous().transpose(1, 2)
    for v in (gaps, turned):
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(rg.quantize_f8(v, "tiles"), (q, s)))


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("m,n,pad", [(1, 1, 0), (130, 260, 200), (300, 513, 0)])
def test_sums_over_rows(rg, counts, m, n, pad, out):  # noqa: F811
    counts = COUNTS[counts]
    e, t = len(counts), sum(counts) + pad
    a, b = normal((t, m), 1, 1.0, torch.bfloat16).cuda(), normal((t, n), 2, 1.0, torch.bfloat16).cuda()
    off = offsets_of(counts)
    (A, SA), (B, SB) = (rg.quantize_f8(x, "columns", offsets=off) for x in (a, b))
    C = rg.grouped_wgrad_f8(A, SA, B, SB, off, out_dtype=out)
    assert C.shape == (e, m, n) and C.dtype == out
    value = lambda q, s: q.double().cpu().numpy() * spread(s.double().cpu().numpy(), 1, 128, q.shape)  # noqa: E731
    av, bv = value(A, SA), value(B, SB)
    for g, c in enumerate(counts):
        at = slice(128 * starts(counts)[g], 128 * starts(counts)[g] + c)
        close(C[g], av[:, at] @ bv[:, at].T, np.abs(av[:, at]) @ np.abs(bv[:, at]).T, blocks(c))
        if not c:
            assert (C[g] == 0).all()
    given = torch.full((e * m * n + 1,), 7.0, dtype=out, device="cuda")
    view = given[1:].view(e, m, n)  # off 16-byte boundaries
    rg.grouped_wgrad_f8(A, SA, B, SB, off, out_dtype=out, out=view)
    assert torch.equal(view, C) and given[0] == 7


def test_sums_over_rows_refuse_bad_offsets(rg):  # noqa: F811
    A, _ = random_f8(20, 256, 1)
    one = torch.ones((20, 2), device="cuda")
    for bad in ([0, 300], [1, 100], [0, -1], [0, 2**40], [0, 200, 100]):
        out = torch.full((len(bad) - 1, 20, 20), 7.0, device="cuda")
        with pytest.raises(rg.ResGemmError) as err:
            rg.grouped_wgrad_f8(A, one, A, one, torch.tensor(bad, device="cuda"), out=out)
        assert err.value.code == rg.RG_ERR_ARG and (out == 7).all()


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------


def expert_inputs(counts, pad, n, k, dtype, seed=0):
    t = sum(counts) + pad
    x, w = normal((t, k), seed + 1, 1.0, dtype), normal((len(counts), n, k), seed + 2, k**-0.5, torch.bfloat16).float()
    return x, w, normal((t, n), seed + 3, 2.0**-4, dtype)


def value(z, rows):
    q, s = quantise_reference(z, rows)
    return q * spread(s, rows, 128, z.shape)


@pytest.mark.parametrize("counts,pad,n,k,dtype", [("ragged", 0, 136, 264, torch.bfloat16),
                                                  ("ragged", 140, 257, 129, torch.float16),
                                                  ("one row", 0, 130, 200, torch.float32),
                                                  ("no rows", 5, 30, 40, torch.bfloat16),
                                                  ("large", 1, 200, 130, torch.bfloat16)])
def test_expert_layer_gradients(rg, counts, pad, n, k, dtype):  # noqa: F811
    counts = COUNTS[counts]
    if dtype == torch.float32:  # entries on a 16-bit grid: the quotient cannot cross an E4M3 tie
        x, w, dy = (v.float() for v in expert_inputs(counts, pad, n, k, torch.bfloat16))
    else:
        x, w, dy = expert_inputs(counts, pad, n, k, dtype)
    Y, saved = rg.expert_linear_f8(x.cuda(), w.cuda(), offsets_of(counts))
    dX, dW = rg.expert_linear_f8_backward(dy.cuda(), saved)
    assert Y.dtype == dX.dtype == dtype and dW.dtype == torch.float32 and dW.shape == w.shape
    xd, wd, dd = x.double().numpy(), w.double().numpy(), dy.double().numpy()
    at = 0
    for g, c in enumerate(counts):
        rows = slice(at, at + c)
        at += c
        if not c:
            assert (dW[g] == 0).all()
            continue
        qw = value(wd[g], 128)
        # scales are fp32: one rounding (2^-24) on each side more than in a product of given scales
        for got, a, b in ((Y[rows], value(xd[rows], 1), qw.T), (dX[rows], value(dd[rows], 1), qw),
                          (dW[g], value(dd[rows].T, 1), value(xd[rows].T, 1).T)):
            close(got, a @ b, np.abs(a) @ np.abs(b), blocks(a.shape[1]), extra=2)
        # against differences of the unquantised product, which is linear in x and in w (bounds as in
        # test_gpu_f8.py: a quantised entry is within 2^-4 of its own or 2^-10 of its scale of the entry)
        off = lambda z, r: np.maximum(np.abs(z) * 2.0**-4, spread(  # noqa: E731
            np.maximum(block_max(z, r, 128), 2.0**-60) / 448.0, r, 128, z.shape) * 2.0**-10)
        v = np.random.default_rng(4).standard_normal(w[g].shape)
        loss = lambda ww: (dd[rows] * (xd[rows] @ ww.T)).sum()  # noqa: E731
        slope = loss(wd[g] + v / 2) - loss(wd[g] - v / 2)
        ed, ex = off(dd[rows].T, 1), off(xd[rows].T, 1).T
        tol = (np.abs(v) * (ed @ np.abs(xd[rows]) + np.abs(dd[rows].T) @ ex + ed @ ex)).sum()
        tol += (np.abs(v) * (2.0**-14 * np.abs(dd[rows].T) @ np.abs(xd[rows]))).sum()
        assert abs((dW[g].double().cpu().numpy() * v).sum() - slope) <= tol
    assert (Y[at:] == 0).all() and (dX[at:] == 0).all()


@pytest.mark.parametrize("dtype,dw", [(torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16),
                                      (torch.float32, torch.float16)])
def test_expert_layer_is_its_parts(rg, dtype, dw):  # noqa: F811
    """The layer's calls give what quantisation and products give one after the other, strided inputs included."""
    counts = [3, 0, 200, 90]
    x = normal((310, 270), 1, 1.0, dtype).cuda()[:, 5:261]
    w = normal((4, 256, 200), 2, 0.1).cuda().transpose(1, 2)  # [4, 200, 256], columns contiguous
    dy = normal((310, 400), 3, 0.01, dtype).cuda()[:, ::2]
    off = offsets_of(counts, torch.int64)
    Y, saved = rg.expert_linear_f8(x, w, off)
    dX, dW = rg.expert_linear_f8_backward(dy, saved, dw_dtype=dw)
    qx, sx, qxt, sxt = rg.quantize_f8(x, "both", offsets=off)
    qw, sw = rg.quantize_f8(w, "tiles")
    qd, sd, qdt, sdt = rg.quantize_f8(dy, "both", offsets=off)
    assert torch.equal(Y, rg.grouped_gemm_f8(qx, sx, qw, sw, off, dtype, transb=True))
    assert torch.equal(dX, rg.grouped_gemm_f8(qd, sd, qw, sw, off, dtype))
    assert torch.equal(dW, rg.grouped_wgrad_f8(qdt, sdt, qxt, sxt, off, dw))


def test_expert_layer_has_a_gradient(rg):  # noqa: F811
    counts, bf = [3, 0, 70, 50], torch.bfloat16
    x, w, dy = (v.cuda() for v in expert_inputs(counts, 9, 96, 200, bf))
    w = w.to(torch.float16)
    off = offsets_of(counts)
    want, saved = rg.expert_linear_f8(x, w, off)
    dx, dw = rg.expert_linear_f8_backward(dy, saved, dw_dtype=w.dtype)
    for needs in ((True, True), (True, False), (False, True)):
        a, b = (t.clone().requires_grad_(n) for t, n in zip((x, w), needs))
        y, _ = rg.expert_linear_f8(a, b, off, sync=False)
        assert y.requires_grad and torch.equal(y, want)
        y.backward(dy)
        for t, n, g in ((a, needs[0], dx), (b, needs[1], dw)):
            assert (t.grad is not None) == n and (not n or (t.grad.dtype == t.dtype and torch.equal(t.grad, g)))
    # offsets that change between the passes are noticed
    b, moved = w.clone().requires_grad_(), off.clone()
    y, _ = rg.expert_linear_f8(x, b, moved)
    moved.add_(1)
    with pytest.raises(RuntimeError):
        y.backward(dy)
    a = x.clone().requires_grad_()
    (grad,) = torch.autograd.grad(rg.expert_linear_f8(a, w, off)[0].sum(), a)  # an expanded gradient
    assert torch.equal(grad, rg.expert_linear_f8_backward(torch.ones_like(want), saved)[0])


def test_expert_layer_reports_bad_offsets(rg):  # noqa: F811
    x, w, dy = (v.cuda() for v in expert_inputs([3, 4], 0, 40, 50, torch.bfloat16))
    y, (kept, off, *rest) = rg.expert_linear_f8(x, w, offsets_of([3, 4]))
    for bad in ([0, 5, 4], [0, 4, 8], [2, 4, 7]):
        bad = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (lambda: rg.expert_linear_f8(x, w, bad),
                     lambda: rg.expert_linear_f8_backward(dy, (kept, bad, *rest))):
            with pytest.raises(rg.ResGemmError) as err:
                call()
            assert err.value.code == rg.RG_ERR_ARG
    with pytest.raises(rg.ResGemmError) as err:
        rg.expert_linear_f8_backward(dy, (kept[:-256], off, *rest))
    assert err.value.code == rg.RG_ERR_WORKSPACE


def test_products_without_a_gradient_do_not_cut_it_silently(rg):  # noqa: F811
    A, _ = random_f8(7, 256, 1)
    B, _ = stack_f8(2, 40, 256, 2)
    off, one = offsets_of([3, 4]), lambda *s: torch.ones(s, device="cuda", requires_grad=True)  # noqa: E731
    for call in (lambda **kw: rg.grouped_gemm_f8(A, one(7, 2), B, one(2, 1, 2), off, transb=True, **kw),
                 lambda **kw: rg.grouped_wgrad_f8(A, one(7, 2), A, one(7, 2), off, **kw)):
        y = call()
        assert y.requires_grad
        with pytest.raises(NotImplementedError):
            y.sum().backward()
        with pytest.raises(ValueError):
            call(out=torch.empty_like(y))


def test_empty(rg):  # noqa: F811
    e = lambda *s: torch.zeros(s, device="cuda").to(F8)  # noqa: E731
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    off = offsets_of([0, 0])
    assert rg.grouped_gemm_f8(e(0, 70), one(0, 1), e(2, 30, 70), one(2, 1, 1), off, transb=True).shape == (0, 30)
    assert rg.grouped_gemm_f8(e(5, 70), one(5, 1), e(2, 70, 0), one(2, 1, 0), off).shape == (5, 0)
    x, w = torch.zeros((0, 40), device="cuda"), torch.ones((2, 30, 40), device="cuda")
    Y, saved = rg.expert_linear_f8(x, w, off)
    dX, dW = rg.expert_linear_f8_backward(Y, saved)
    assert Y.shape == (0, 30) and dX.shape == (0, 40) and dW.shape == (2, 30, 40) and (dW == 0).all()


def test_timeout_is_reported(rg, variant):  # noqa: F811
    """A product whose tensor-core stage never reports its first block ends with a time-out, and the next is sound."""
    lib = rg.library()
    A, SA, B, SB, good = check_rows(rg, [200, 100], 512, 512, True, torch.float32)
    old = lib.rg_set_wait_limit_ns(50_000_000)
    try:
        lib.rg_inject_fault(1)
        with pytest.raises(rg.ResGemmError) as err:
            rg.grouped_gemm_f8(A, SA, B, SB, offsets_of([200, 100]), torch.float32, True)
        assert err.value.code == rg.RG_ERR_TIMEOUT
    finally:
        lib.rg_inject_fault(0)
        lib.rg_set_wait_limit_ns(old)
    assert torch.equal(rg.grouped_gemm_f8(A, SA, B, SB, offsets_of([200, 100]), torch.float32, True), good)


# ---------------------------------------------------------------------------
# results of more than 2^31 entries
# ---------------------------------------------------------------------------


def test_rows_of_many_entries(rg, variant):  # noqa: F811
    """The last rows of a result whose entries pass 2^31, and the rows behind the last group."""
    t, n, counts = 70000, 32768, [30000, 39990]
    A, a = random_f8(t, 16, 1)
    B, b = stack_f8(2, n, 16, 2)
    SA, sa = random_scales((t, 1), 3)
    SB, sb = random_scales((2, n // 128, 1), 4)
    C = rg.grouped_gemm_f8(A, SA, B, SB, offsets_of(counts), torch.bfloat16, True)
    rows = np.r_[0:3, 29998:30003, 65530:65540, 69980:69990]
    for r in rows:
        g = int(r >= 30000)
        bv = b[g] * np.repeat(sb[g], 128, 0)
        av = a[r] * sa[r]
        close(C[r], bv @ av, np.abs(bv) @ np.abs(av), 1)
    assert (C[69990:] == 0).all()


def test_sums_of_many_entries(rg):  # noqa: F811
    m, counts = 8192, [3] * 40
    x = normal((120, m), 1, 1.0, torch.bfloat16).cuda()
    off = offsets_of(counts)
    A, SA = rg.quantize_f8(x, "columns", offsets=off)
    C = rg.grouped_wgrad_f8(A, SA, A, SA, off, out_dtype=torch.bfloat16)
    av = A.double().cpu().numpy() * spread(SA.double().cpu().numpy(), 1, 128, A.shape)
    for g in (0, 31, 32, 39):
        at = slice(128 * starts(counts)[g], 128 * starts(counts)[g] + 3)
        for r in (0, 4095, 8191):
            close(C[g, r], av[:, at] @ av[r, at], np.abs(av[:, at]) @ np.abs(av[r, at]), 1)
