"""The expert layer where its products split k over warps, where few tokens fit into a pass, and how exactly the gated
product enters the second product.  Bounds as in test_gpu_f8.py."""
import numpy as np
import pytest
import torch

from gpu_util import rg  # noqa: F401
from test_gpu_f8 import F8, U, blocks

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
