"""The 8-bit block-scaled operators together, as a model uses them: train a linear layer, then decode with experts.

    python examples/f8_layers.py

1. A linear layer fits a target by gradient descent: its output and both gradients are 8-bit products
   (linear_f8, whose gradient is linear_f8_backward), its weights stay float32.
2. The trained weights are quantised once (quantize_f8, 128 x 128 tiles) and serve single tokens with
   scaled_gemm_f8, and a mixture-of-experts layer with 8-bit weights decodes the same tokens (moe_layer_f8).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import exact_modular_int8_gb300 as rg  # noqa: E402


def train(steps=40, tokens=512, features=384, outputs=256, seed=0):
    """(losses, weights) of a layer that learns another layer's outputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    target = torch.randn((outputs, features), generator=g, device="cuda") * features**-0.5
    w = torch.zeros((outputs, features), device="cuda", requires_grad=True)
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, features), generator=g, device="cuda").to(torch.bfloat16)
        want = x.float() @ target.t()
        y, _ = rg.linear_f8(x, w, sync=False)
        loss = (y.float() - want).square().mean()
        loss.backward()
        with torch.no_grad():
            w -= 100.0 * w.grad
            w.grad = None
        losses.append(loss.detach())
    return [float(v) for v in losses], w.detach()


def decode(w, tokens=3, experts=16, hidden=384, inner=512, top_k=4, seed=1):
    """(layer outputs, expert outputs) for a few tokens, with all weights in 8 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").to(torch.bfloat16)
    router = (torch.randn((experts, hidden), generator=g, device="cuda") * hidden**-0.5).to(torch.bfloat16)

    def expert_weights(n, k):
        parts = [rg.quantize_f8(torch.randn((n, k), generator=g, device="cuda") * k**-0.5, "tiles")
                 for _ in range(experts)]
        return torch.stack([q.view(torch.uint8) for q, _ in parts]).view(rg.f8.F8), torch.stack([s for _, s in parts])

    w13, s13 = expert_weights(2 * inner, hidden)
    w2, s2 = expert_weights(hidden, inner)
    qw, sw = rg.quantize_f8(w, "tiles")
    qx, sx = rg.quantize_f8(x, "rows", sync=False)
    y = rg.scaled_gemm_f8(qx, sx, qw, sw, transb=True, sync=False)
    return y, rg.moe_layer_f8(x, router, w13, s13, w2, s2, top_k)


if __name__ == "__main__":
    losses, weights = train()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.6f} in {len(losses)} steps")
    y, z = decode(weights)
    print("decoded", tuple(y.shape), tuple(z.shape), "finite:", bool(torch.isfinite(y).all() and torch.isfinite(z).all()))
