"""Forms of the 8-bit product and quantisation beside those of test_gpu_f8.py: every shape of the few-row kernel, walks
over several tiles of a block, and fp32 entries of all 24 bits.  Bounds as there."""
import numpy as np
import pytest
import torch

from gpu_util import rg  # noqa: F401
from test_gpu_f8 import GRID, block_max, check_product, nearest_e4m3, spread

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("n,k", [(33, 100), (129, 1025), (515, 2000)])
@pytest.mark.parametrize("m", [2, 8, 9, 16, 17, 24, 25, 32])
def test_few_rows(rg, m, n, k, tile):  # noqa: F811
    check_product(rg, m, n, k, True, tile, torch.float32, seed=m)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m", [12, 31])
def test_few_rows_16_bit_results(rg, m, out):  # noqa: F811
    check_product(rg, m, 391, 640, True, True, out, seed=m)


@pytest.mark.parametrize("m,n,k,tile", [(1, 20000, 1300, True), (12, 20000, 1300, False), (12, 40001, 1030, True),
                                        (20, 3100, 1300, True), (32, 4001, 1040, False), (7, 20000, 1111, False)])
def test_few_rows_over_many_tiles(rg, m, n, k, tile):  # noqa: F811
    """More tiles than blocks and more 128-blocks than warps: pieces are copied ahead from one tile to the next."""
    check_product(rg, m, n, k, True, tile, torch.float32, seed=7)


@pytest.mark.parametrize("form,rows,turned", [("rows", 1, False), ("columns", 1, True), ("both", 1, True),
                                              ("tiles", 128, False)])
@pytest.mark.parametrize("m,k", [(1, 4096), (130, 391), (257, 1032), (300, 14000)])
def test_quantise_whole_fp32_entries(rg, form, rows, turned, m, k):  # noqa: F811
    """fp32 entries of 24 bits.  448 x / a is formed in fp32 (x 0.875 rounded, then a correctly rounded quotient:
    within 2^-23 of itself) and rounded to E4M3 from there, so a value is the nearest one, or a neighbour of a quotient
    that close to the middle between the two."""
    x = torch.from_numpy(np.random.default_rng(m + k).standard_normal((m, k)).astype(np.float32) * np.float32(3))
    got = rg.quantize_f8(x.cuda(), form)
    xd = x.double().numpy()
    pairs = [(xd, got[0], got[1])] if form != "columns" else []
    pairs += [(xd.T, got[-2], got[-1])] if turned else []
    for z, q, s in pairs:
        a = block_max(z, rows, 128)
        np.testing.assert_array_equal(s.cpu().numpy(), (a / 448.0).astype(np.float32))
        v = z * 448.0 / spread(a, rows, 128, z.shape)
        q, want = q.float().double().cpu().numpy(), nearest_e4m3(v)
        at = np.searchsorted(GRID, np.abs(v)).clip(1, 126)
        middle = (GRID[at - 1] + GRID[at]) / 2
        near = np.abs(np.abs(v) - middle) <= 2.0**-22 * np.abs(v)
        other = np.sign(v) * np.where(np.abs(want) == GRID[at], GRID[at - 1], GRID[at])
        assert ((q == want) | (near & (q == other))).all()
        assert (q != want).mean() < 1e-4
