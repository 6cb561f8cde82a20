"""Training steps of the 8-bit layers at the ends of their ranges: infinite values before an activation, sums over rows
on both sides of a cluster, gradients that are not wanted, offsets that change between the passes, captures."""
import math

import pytest
import torch

from gpu_util import rg  # noqa: F401
from test_gpu_f8 import normal
from test_gpu_f8_act import ACTS, layer_inputs

pytestmark = pytest.mark.gpu
bf, f16, f32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,big", [(f16, 7e4), (f16, math.inf), (bf, math.inf), (f32, math.inf)])
def test_slopes_of_infinite_values(rg, dtype, big, act):  # noqa: F811
    """Values before the activation that are kept as infinities (fp16: finite ones beyond 65504) have the slopes of
    large ones, 0 or 1, and leave every gradient finite."""
    m, n, k = 150, 200, 72
    x, w, b, dy = layer_inputs(m, n, k, dtype)
    b = b.float()
    b[::5], b[2::7] = -big, big
    near = b.clamp(-6e4, 6e4)
    _, saved = rg.linear_act_f8(x, w, bias=b, act=act)
    got = rg.linear_act_f8_backward(dy, saved)
    _, saved = rg.linear_act_f8(x, w, bias=near, act=act)
    for g, want in zip(got, rg.linear_act_f8_backward(dy, saved)):
        assert torch.isfinite(g).all() and torch.equal(g, want)
    ref = dy.double().sum(0)
    tol = (m / 8 + 24) * 2.0**-24 * dy.double().abs().sum(0)
    assert ((got[2] - ref).abs() <= tol)[2::7].all()
    if act is not None:
        gone = torch.ones(n, dtype=torch.bool)[::5]
        gone[[i for i in range(len(gone)) if (5 * i) % 7 == 2]] = False  # overwritten by +big
        assert (got[2][::5][gone] == 0).all()


def test_status_of_two_products_at_once(rg):  # noqa: F811
    """The weight gradient's kernel may run beside the input gradient's, whose first block clears the status for both:
    what either reports stays."""
    x, w, dy = normal((40, 128), 1, 1.0, bf).cuda(), normal((2, 96, 128), 2, 0.1).cuda(), normal((40, 96), 3, 1.0, bf).cuda()
    off = torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")
    ws = torch.empty(rg.library().expert_linear_f8_ws_bytes(40, 96, 128, 2), dtype=torch.uint8, device="cuda")
    _, (kept, _, *rest) = rg.expert_linear_f8(x, w, off, ws=ws)
    bad = torch.tensor([0, 50, 40], dtype=torch.int32, device="cuda")
    for i in range(100):
        at, code = (bad, rg.RG_ERR_ARG) if i % 3 else (off, rg.RG_OK)
        rg.expert_linear_f8_backward(dy, (kept, at, *rest), sync=False, ws=ws)
        assert rg.status(ws) == code
