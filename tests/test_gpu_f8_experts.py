"""The expert layer where its products split k over warps, where few tokens fit into a pass, and how exactly the gated
product enters the second product.  Bounds as in test_gpu_f8.py."""
import numpy as np
import pytest
import torch

from gpu_util import rg  # noqa: F401
from test_gpu_f8 import F8, U, blocks, check_moe, moe_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("i", [64, 272, 2064])
@pytest.mark.parametrize("t", [3, 13])
def test_gated_product_keeps_its_low_bits(rg, t, i, dtype):  # noqa: F811
    """Each output is the difference of two entries of the gated product that agree in their first 12 bits, so what it
    shows is the bits below.  The error: an entry of h takes silu (8 units) and two rounded factors, and enters the
    second product within 2^-23 of itself or 2^-39 of the row's largest; the product's sums as in a product."""
    h, u = 32, 2.0**-23
    r = np.random.default_rng(i + t)
    x = np.zeros((t, h))
    x[:, 0] = 1 + r.integers(0, 128, t) / 128
    x[:, 1] = 2.0**-13 * (1 + r.integers(0, 128, t) / 128)
    w13, w2 = np.zeros((1, 2 * i, h)), np.zeros((1, h, i))
    w13[0, :i, 0] = 1.0
    w13[0, i:, 0] = np.repeat(1 + r.integers(0, 8, i // 2) / 8, 2)
    w13[0, i + 1 :: 2, 1] = 1 + r.integers(0, 8, i // 2) / 8
    pair = r.permutation(i // 2)[:h]
    out = np.arange(len(pair))
    w2[0, out, 2 * pair], w2[0, out, 2 * pair + 1] = -1.0, 1.0
    a, b = x @ w13[0, :i].T, x @ w13[0, i:].T
    g = a / (1 + np.exp(-a)) * b
    y, mag = g @ w2[0].T, np.abs(g) @ np.abs(w2[0]).T
    eh = 12 * u * np.abs(g) + 2.0**-39 * np.abs(g).max(1, keepdims=True)
    err = eh @ np.abs(w2[0]).T + (8 * 17 + blocks(i) + 12) * u * mag
    f8 = lambda w: torch.from_numpy(w).float().to(F8).cuda()  # noqa: E731
    one = lambda n, k: torch.ones((1, blocks(n), blocks(k)), device="cuda")  # noqa: E731
    Y = rg.moe_layer_f8(torch.from_numpy(x).to(dtype).cuda(), torch.zeros((1, h), dtype=dtype, device="cuda"), f8(w13),
                        one(2 * i, h), f8(w2), one(h, i), 1)
    got = Y.double().cpu().numpy()
    assert (np.abs(got - y) <= err + U[dtype] * (np.abs(y) + err) + 2.0**-25).all(), np.abs(got - y).max()


def test_overflowed_gated_product(rg):  # noqa: F811
    """A gated product that leaves fp32's range in one place: outputs that take it are inf with the sign of its weight
    (the other, finite entries must not become inf too and make them NaN)."""
    t, h, i = 5, 32, 144
    x = torch.zeros((t, h), dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = 2.0**60, 2.0**40
    w13, w2 = torch.zeros((1, 2 * i, h)), torch.zeros((1, h, i))
    w13[0, 7, 0] = w13[0, i + 7, 0] = 256.0  # h[7] = 2^136
    w13[0, 130, 0], w13[0, i + 130, 1] = 1.0, 1.0  # h[130] = 2^100
    w13[0, 131, 1] = w13[0, i + 131, 1] = 1.0  # h[131] = 2^80
    w2[0, :, 7] = torch.tensor([1.0, -1.0] * (h // 2))
    w2[0, :, 130] = -w2[0, :, 7]
    w2[0, :, 131] = -2.0 * w2[0, :, 7]
    one = lambda n, k: torch.ones((1, blocks(n), blocks(k)), device="cuda")  # noqa: E731
    Y = rg.moe_layer_f8(x.cuda(), torch.zeros((1, h), dtype=torch.bfloat16, device="cuda"), w13.to(F8).cuda(),
                        one(2 * i, h), w2.to(F8).cuda(), one(h, i), 1)
    assert torch.equal(Y.float().cpu(), (w2[0, :, 7] * float("inf")).expand(t, h))


# Widths of 16 blocks of 128 and more split k over warps (2048: two of them, 4096: four, 8192: eight); 16 tokens
# on one expert take two column tiles, and tokens of 16384 and more entries fit a few at a time, so that an expert takes
# several passes.
@pytest.mark.parametrize("t,h,i,e,top_k,renorm,dtype", [
    (3, 2048, 2064, 4, 2, True, torch.bfloat16), (13, 2048, 2064, 1, 1, True, torch.float16),
    (16, 1936, 80, 1, 1, False, torch.bfloat16), (17, 4112, 272, 3, 1, True, torch.bfloat16),
    (9, 272, 8208, 2, 1, False, torch.float16), (64, 2064, 144, 5, 2, True, torch.bfloat16),
    (17, 16384, 32, 1, 1, True, torch.bfloat16), (5, 32768, 48, 1, 1, True, torch.float16),
    (6, 48, 16400, 1, 1, True, torch.bfloat16), (3, 64, 24960, 1, 1, True, torch.bfloat16),
    (3, 64, 24976, 1, 1, True, torch.float16), (4, 48, 32768, 1, 1, True, torch.bfloat16)])
def test_wide_layers(rg, t, h, i, e, top_k, renorm, dtype):  # noqa: F811
    check_moe(rg, moe_inputs(t, h, i, e, dtype, 17 * t + h + i), top_k, renorm)


@pytest.mark.parametrize("h,i", [(2048, 2048), (4096, 1040)])
def test_a_token_alone_and_in_a_batch_of_a_wide_layer(rg, h, i):  # noqa: F811
    """Equal calls give equal bits, and a token's result does not depend on what comes with it."""
    args = [a.cuda() for a in moe_inputs(16, h, i, 3, torch.bfloat16, h + i)]
    Y = rg.moe_layer_f8(*args, 2)
    for _ in range(3):
        assert torch.equal(rg.moe_layer_f8(*args, 2), Y)
    for t in range(16):
        assert torch.equal(rg.moe_layer_f8(args[0][t : t + 1], *args[1:], 2)[0], Y[t])
