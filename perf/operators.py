"""What the 8-bit block-scaled operators are measured on: quantisation, product, linear layer and expert layer.

All four share one number format: E4M3 values with one fp32 scale for every 128 values along the contraction
(activations and gradients) or for every 128 x 128 tile (weights); a value stands for q * s.

  quantize  16- or 32-bit matrix -> E4M3 values and scales
  gemm      the product of two such matrices, in the directions a linear layer needs (forward, input gradient,
            weight gradient)
  linear    a linear layer's training step from 16-bit tensors: output, input gradient, weight gradient
  moe       a whole mixture-of-experts layer for a few tokens: router, top-k, gated experts, weighted sum

`own` chooses between the plain form (elementary torch operations in 32 bits, rounded once at the end) and the
library's entry points.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0**-60  # a block whose largest magnitude is below this is scaled as if it were this
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # One token's activations before a product: pure latency.
        {"name": "quantize rows 1 token", "op": "quantize", "form": "rows", "dtype": "bf16", "m": 1, "k": 4096},
        # A training batch's activations, for the output (along rows) and for the weight gradient (along columns);
        # a ragged number of tokens and of features.
        {"name": "quantize both 8100x4104", "op": "quantize", "form": "both", "dtype": "bf16", "m": 8100, "k": 4104},
        # Serving, one token through one weight matrix: the weights are read once.
        {"name": "gemm 1x4096x2048", "op": "gemm", "way": "forward", "m": 1, "n": 4096, "k": 2048, "out": "bf16"},
        # Serving a small batch.
        {"name": "gemm 24x8192x4096", "op": "gemm", "way": "forward", "m": 24, "n": 8192, "k": 4096, "out": "bf16"},
        # The input gradient at ragged sizes: the weights are read in the order in which they are stored, [N, K].
        {"name": "gemm dgrad 1000x1544x2056", "op": "gemm", "way": "dgrad", "m": 1000, "n": 1544, "k": 2056,
         "out": "bf16"},
        # The weight gradient: one scale per 128 on both sides, fp32 sums out, a ragged number of tokens.
        {"name": "gemm wgrad 2048x4096x8100", "op": "gemm", "way": "wgrad", "m": 2048, "n": 4096, "k": 8100,
         "out": "f32"},
        # Prefill or training at full size: the tensor cores' rate counts.
        {"name": "gemm 8192x8192x4096", "op": "gemm", "way": "forward", "m": 8192, "n": 8192, "k": 4096,
         "out": "bf16"},
        # A small layer's training step: many short launches.
        {"name": "linear step 512x1024x1024", "op": "linear", "m": 512, "n": 1024, "k": 1024},
        # A large layer's training step.
        {"name": "linear step 8192x4096x4096", "op": "linear", "m": 8192, "n": 4096, "k": 4096},
        # Decoding one token through an expert layer: 8 of 64 experts' weights are read.
        {"name": "moe 1 token", "op": "moe", "t": 1, "h": 2048, "i": 1024, "e": 64, "top_k": 8, "renorm": True},
        # A few sequences decode together; ragged widths, few large experts, unnormalised weights.
        {"name": "moe 7 tokens", "op": "moe", "t": 7, "h": 1808, "i": 1552, "e": 16, "top_k": 2, "renorm": False},
        # The largest batch of "a few tokens": nearly all experts' weights are read.
        {"name": "moe 64 tokens", "op": "moe", "t": 64, "h": 4096, "i": 1024, "e": 128, "top_k": 8, "renorm": True},
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["quantize", "gemm", "gemm", "gemm", "linear", "moe", "moe"])
    if op == "quantize":
        m = size(1, 8192)
        return {"op": op, "form": rng.choice(["rows", "columns", "both", "tiles"]),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "m": m, "k": size(64, 4096)}
    if op == "gemm":
        return {"op": op, "way": rng.choice(["forward", "dgrad", "wgrad"]), "m": size(1, 8192), "n": size(64, 8192),
                "k": size(100, 4096), "out": rng.choice(["bf16", "f16", "f32"])}
    if op == "linear":
        return {"op": op, "m": size(64, 8192), "n": size(128, 4096), "k": size(128, 4096)}
    e = size(8, 128)
    return {"op": op, "t": size(1, 64), "h": 16 * size(16, 256), "i": 16 * size(8, 64), "e": e,
            "top_k": rng.randint(1, 8), "renorm": rng.random() < 0.5}


def work(case):
    blocks = lambda x: -(-x // BLOCK)  # noqa: E731
    if case["op"] == "quantize":
        m, k, form = case["m"], case["k"], case["form"]
        b = m * k * (4 if case["dtype"] == "f32" else 2) + m * k * (2 if form == "both" else 1)
        b += 4 * {"rows": m * blocks(k), "columns": k * blocks(m), "both": m * blocks(k) + k * blocks(m),
                  "tiles": blocks(m) * blocks(k)}[form]
        return {"bytes": b, "flops": 2 * m * k * (2 if form == "both" else 1)}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        b = m * k + n * k + m * n * (4 if case["out"] == "f32" else 2) + 4 * m * blocks(k)
        b += 4 * blocks(k) * (n if case["way"] == "wgrad" else blocks(n))
        return {"bytes": b, "flops": 2 * m * n * k}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        # x, dy (16 bits), w (32 bits) in; y, dx (16 bits), dw (32 bits) out
        return {"bytes": 2 * (m * k + m * n) + 4 * n * k + 2 * (m * n + m * k) + 4 * n * k, "flops": 6 * m * n * k}
    t, h, i, e, k = (case[x] for x in ("t", "h", "i", "e", "top_k"))
    used = e * (1 - (1 - k / e) ** t)  # experts that some token chooses, for even routing
    return {"bytes": int(used * 3 * h * i) + 2 * e * h + 4 * t * h, "flops": 2 * t * k * 3 * h * i + 2 * t * e * h}


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------


def spread(s, rows, cols, shape):
    """Scales repeated over their blocks of `rows` x `cols` entries, cut to `shape`."""
    return s.repeat_interleave(rows, -2).repeat_interleave(cols, -1)[..., : shape[-2], : shape[-1]]


def block_amax(x, rows, cols):
    """Largest magnitudes of the blocks of a matrix (missing entries count as 0)."""
    m, k = x.shape
    mb, kb = -(-m // rows), -(-k // cols)
    x = torch.nn.functional.pad(x.abs(), (0, kb * cols - k, 0, mb * rows - m))
    return x.view(mb, rows, kb, cols).amax((1, 3))


def plain_quantize(x, rows, cols):
    """E4M3 values and scales with one scale for each block of rows x cols entries: s = amax / 448, and q = 448 x / amax
    rounded to the nearest E4M3 value (the factor split into 0.875 and 512, so that neither side overflows and the
    products of 16-bit entries are exact)."""
    x = x.float()
    a = block_amax(x, rows, cols).clamp_min(TINY)
    q = (x * 0.875) / spread(a * 2.0**-9, rows, cols, x.shape)
    return q.to(torch.float8_e4m3fn), a / E4M3_MAX


def plain_value(q, s, rows, cols):
    return q.float() * spread(s, rows, cols, q.shape)


def plain_linear(x, w, dy):
    qx, sx = plain_quantize(x, 1, BLOCK)
    qw, sw = plain_quantize(w, BLOCK, BLOCK)
    qd, sd = plain_quantize(dy, 1, BLOCK)
    qxt, sxt = plain_quantize(x.t(), 1, BLOCK)
    qdt, sdt = plain_quantize(dy.t(), 1, BLOCK)
    w8 = plain_value(qw, sw, BLOCK, BLOCK)
    y = plain_value(qx, sx, 1, BLOCK) @ w8.t()
    dx = plain_value(qd, sd, 1, BLOCK) @ w8
    dw = plain_value(qdt, sdt, 1, BLOCK) @ plain_value(qxt, sxt, 1, BLOCK).t()
    return y.to(x.dtype), dx.to(x.dtype), dw


def plain_moe(x, wr, w13, s13, w2, s2, top_k, renorm):
    t, h = x.shape
    e, i = w13.shape[0], w2.shape[2]
    xf = x.float()
    p = torch.softmax(xf @ wr.float().t(), 1)
    g, idx = torch.sort(p, dim=1, descending=True, stable=True)
    g, idx = g[:, :top_k], idx[:, :top_k]
    if renorm:
        g = g / g.sum(1, keepdim=True)
    if t * top_k <= e:  # fewer choices than experts: gather the chosen experts' weights
        f = idx.reshape(-1)
        a = plain_value(w13[f], s13[f], BLOCK, BLOCK) @ xf.repeat_interleave(top_k, 0).unsqueeze(2)
        a = a.squeeze(2)
        z = a[:, :i] / (1 + torch.exp(-a[:, :i])) * a[:, i:]
        y = (plain_value(w2[f], s2[f], BLOCK, BLOCK) @ z.unsqueeze(2)).view(t, top_k, h)
        return (y * g.unsqueeze(2)).sum(1).to(x.dtype)
    full = torch.zeros((t, e), device=x.device).scatter_(1, idx, g)  # every expert, weighted by 0 where not chosen
    a = xf.unsqueeze(0) @ plain_value(w13, s13, BLOCK, BLOCK).transpose(1, 2)
    z = a[..., :i] / (1 + torch.exp(-a[..., :i])) * a[..., i:]
    y = z @ plain_value(w2, s2, BLOCK, BLOCK).transpose(1, 2)
    return (y * full.t().unsqueeze(2)).sum(0).to(x.dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def rows16(q):
    """The same matrix with rows that start on 16-byte boundaries, as quantised matrices are stored."""
    m, k = q.shape
    buf = torch.zeros((m, -(-k // 16) * 16), dtype=torch.uint8, device=q.device).view(q.dtype)
    buf[:, :k] = q
    return buf[:, :k]


def activations(g, m, k, dtype):
    """Normal entries, with some features much larger than the others, as hidden states have them."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn((1, k), generator=g, device="cuda"))
    return x.to(dtype)


def weights(g, *shape):
    return torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5


def expert_weights(g, e, n, k):
    """[E, N, K] E4M3 weights and their [E, ceil(N / 128), ceil(K / 128)] scales, quantised a few experts at a time."""
    step = max(1, (1 << 28) // (n * k))
    q, s = [], []
    for e0 in range(0, e, step):
        c = min(step, e - e0)
        nb, kb = -(-n // BLOCK), -(-k // BLOCK)
        w = weights(g, c, n, k)
        a = torch.nn.functional.pad(w.abs(), (0, kb * BLOCK - k, 0, nb * BLOCK - n))
        sc = a.view(c, nb, BLOCK, kb, BLOCK).amax((2, 4)).clamp_min(TINY) / E4M3_MAX
        q.append((w * spread(1.0 / sc, BLOCK, BLOCK, w.shape)).to(torch.float8_e4m3fn).view(torch.uint8))
        s.append(sc)
    return torch.cat(q).view(torch.float8_e4m3fn), torch.cat(s)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    if case["op"] == "quantize":
        st["x"] = activations(g, case["m"], case["k"], DTYPES[case["dtype"]])
    elif case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        qa, st["sa"] = plain_quantize(activations(g, m, k, torch.float32), 1, BLOCK)
        if case["way"] == "forward":  # weights [N, K]
            qb, st["sb"] = plain_quantize(weights(g, n, k), BLOCK, BLOCK)
        elif case["way"] == "dgrad":  # weights [K, N]: the contraction runs over their rows
            qb, st["sb"] = plain_quantize(weights(g, k, n), BLOCK, BLOCK)
        else:  # another activation-like operand [N, K]
            qb, st["sb"] = plain_quantize(activations(g, n, k, torch.float32), 1, BLOCK)
        st["a"], st["b"] = rows16(qa), rows16(qb)
    elif case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"] = activations(g, m, k, torch.bfloat16)
        st["w"] = weights(g, n, k)
        st["dy"] = activations(g, m, n, torch.bfloat16) * 1e-3
    else:
        st["x"] = activations(g, case["t"], case["h"], torch.bfloat16)
        st["wr"] = weights(g, case["e"], case["h"]).to(torch.bfloat16)
        st["w13"], st["s13"] = expert_weights(g, case["e"], 2 * case["i"], case["h"])
        st["w2"], st["s2"] = expert_weights(g, case["e"], case["h"], case["i"])
    if own:
        import exact_modular_int8_gb300 as rg

        rg.library()
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(st):
    if own:
        import exact_modular_int8_gb300 as rg

        if st["op"] == "quantize":
            return rg.quantize_f8(st["x"], st["form"], sync=False)
        if st["op"] == "gemm":
            return rg.scaled_gemm_f8(st["a"], st["sa"], st["b"], st["sb"], out_dtype=DTYPES[st["out"]],
                                     transb=st["way"] != "dgrad", sync=False)
        if st["op"] == "linear":
            y, saved = rg.linear_f8(st["x"], st["w"], sync=False)
            dx, dw = rg.linear_f8_backward(st["dy"], saved, sync=False)
            return y, dx, dw
        return rg.moe_layer_f8(st["x"], st["wr"], st["w13"], st["s13"], st["w2"], st["s2"], st["top_k"],
                               renorm=st["renorm"], sync=False)
    if st["op"] == "quantize":
        x, form = st["x"], st["form"]
        if form == "tiles":
            return plain_quantize(x, BLOCK, BLOCK)
        out = plain_quantize(x, 1, BLOCK) if form in ("rows", "both") else ()
        return out + (plain_quantize(x.t(), 1, BLOCK) if form in ("columns", "both") else ())
    if st["op"] == "gemm":
        a = plain_value(st["a"], st["sa"], 1, BLOCK)
        b = plain_value(st["b"], st["sb"], 1 if st["way"] == "wgrad" else BLOCK, BLOCK)
        return (a @ (b if st["way"] == "dgrad" else b.t())).to(DTYPES[st["out"]])
    if st["op"] == "linear":
        return plain_linear(st["x"], st["w"], st["dy"])
    return plain_moe(*(st[x] for x in ("x", "wr", "w13", "s13", "w2", "s2", "top_k", "renorm")))


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------


def exact_quantize(x, rows):
    """(q, s) in 64 bits; rows = 1 or 128 rows to a block of 128 columns."""
    x = x.double()
    m, k = x.shape
    q, s = torch.empty_like(x), x.new_empty((-(-m // rows), -(-k // BLOCK)))
    for j in range(s.shape[1]):
        part = x[:, j * BLOCK : (j + 1) * BLOCK]
        top = part.abs().max(1).values
        if rows > 1:
            pad = torch.zeros(s.shape[0] * rows, dtype=torch.float64, device=x.device)
            pad[:m] = top
            top = pad.view(-1, rows).max(1).values
        s[:, j] = torch.maximum(top, torch.full_like(top, TINY)) / E4M3_MAX
        v = part * E4M3_MAX / torch.maximum(top, torch.full_like(top, TINY)).repeat_interleave(rows)[:m, None]
        # E4M3: three stored significand bits, exponents from -6 up
        step = torch.exp2(torch.frexp(v)[1].clamp_min(-5).double() - 4)
        q[:, j * BLOCK : (j + 1) * BLOCK] = torch.round(v / step) * step
    return q, s


def exact_product(a, sa, b, sb, rows_b):
    """Sum over blocks of 128 of (a_block b_block^T) weighted by both sides' scales; b is [N, K]."""
    out = torch.zeros((a.shape[0], b.shape[0]), dtype=torch.float64, device=a.device)
    for j in range(sa.shape[1]):
        at = slice(j * BLOCK, (j + 1) * BLOCK)
        col = sb[:, j].double().repeat_interleave(rows_b)[: b.shape[0]]
        out += (a[:, at].double() @ b[:, at].double().t()) * sa[:, j].double()[:, None] * col[None, :]
    return out


def exact_moe(st):
    x, i, k = st["x"].double(), st["i"], st["top_k"]
    logits = x @ st["wr"].double().t()
    p = torch.exp(logits - logits.max(1, keepdim=True).values)
    p /= p.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    chosen = torch.zeros_like(p, dtype=torch.bool)
    rest = p.clone()
    for _ in range(k):
        at = rest.argmax(1)
        chosen[torch.arange(len(at), device=at.device), at] = True
        rest[torch.arange(len(at), device=at.device), at] = -1
    p = torch.where(chosen, p, torch.zeros_like(p))
    if st["renorm"]:
        p = p / p.sum(1, keepdim=True)
    for e in chosen.any(0).nonzero().flatten().tolist():
        who = chosen[:, e].nonzero().flatten()
        w13 = st["w13"][e].double() * spread(st["s13"][e].double(), BLOCK, BLOCK, st["w13"][e].shape)
        w2 = st["w2"][e].double() * spread(st["s2"][e].double(), BLOCK, BLOCK, st["w2"][e].shape)
        a = x[who] @ w13.t()
        y[who] += p[who, e][:, None] * ((a[:, :i] * torch.sigmoid(a[:, :i]) * a[:, i:]) @ w2.t())
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        x, form = st["x"], case["form"]
        if form == "tiles":
            return exact_quantize(x, BLOCK)
        out = exact_quantize(x, 1) if form in ("rows", "both") else ()
        return out + (exact_quantize(x.t(), 1) if form in ("columns", "both") else ())
    if case["op"] == "gemm":
        b, sb = (st["b"].t(), st["sb"].t()) if case["way"] == "dgrad" else (st["b"], st["sb"])
        return exact_product(st["a"], st["sa"], b, sb, 1 if case["way"] == "wgrad" else BLOCK)
    if case["op"] == "linear":
        w, sw = exact_quantize(st["w"], BLOCK)
        y = exact_product(*exact_quantize(st["x"], 1), w, sw, BLOCK)
        dx = exact_product(*exact_quantize(st["dy"], 1), w.t(), sw.t(), BLOCK)
        dw = exact_product(*exact_quantize(st["dy"].t(), 1), *exact_quantize(st["x"].t(), 1), 1)
        return y, dx, dw
    return exact_moe(st)
