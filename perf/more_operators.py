"""What the 8-bit products with an epilogue and the products grouped by expert are measured on.

The number format is that of the other 8-bit operators: E4M3 values with one fp32 scale for every 128 values along the
contraction (activations and gradients) or for every 128 x 128 tile (weights); a value stands for q * s.

  experts   products grouped by expert: rows sorted by expert, a weight matrix each, in the directions a layer needs
            (output, input gradient, weight gradient)
  step      an expert layer's training step from 16-bit tensors: output, input gradient, weight gradients
  act       a product with bias, activation and residual in its epilogue
  act step  the training step of a linear layer with bias, activation and residual

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
        # One token decodes through the first product of an expert layer: 8 of 64 experts get a row each.
        {"name": "experts 1 token", "op": "experts", "way": "forward", "t": 1, "top_k": 8, "e": 64, "n": 2048,
         "k": 2048, "pad": 0, "out": "bf16"},
        # A batch of sequences decodes: nearly every expert's weights are read for a few rows each.
        {"name": "experts 64 tokens", "op": "experts", "way": "forward", "t": 64, "top_k": 8, "e": 64, "n": 2048,
         "k": 4096, "pad": 0, "out": "bf16"},
        # A prompt or a training batch: the tensor cores' rate counts.
        {"name": "experts 8192 tokens", "op": "experts", "way": "forward", "t": 8192, "top_k": 8, "e": 64, "n": 2048,
         "k": 4096, "pad": 0, "out": "bf16"},
        # The input gradient at ragged sizes, in a buffer of fixed capacity: rows behind the last group.
        {"name": "experts dgrad 1250 tokens", "op": "experts", "way": "dgrad", "t": 1250, "top_k": 4, "e": 16,
         "n": 1544, "k": 2056, "pad": 120, "out": "bf16"},
        # The weight gradients: a short, ragged contraction for each expert and much to write.
        {"name": "experts wgrad 4096 tokens", "op": "experts", "way": "wgrad", "t": 4096, "top_k": 4, "e": 32,
         "n": 2048, "k": 2048, "pad": 0, "out": "f32"},
        # A small expert layer's training step: many short launches.
        {"name": "step 512 tokens", "op": "step", "t": 512, "top_k": 2, "e": 8, "n": 1024, "k": 1024, "pad": 0},
        # A large expert layer's training step.
        {"name": "step 8192 tokens", "op": "step", "t": 8192, "top_k": 4, "e": 16, "n": 2048, "k": 4096, "pad": 0},
        # Decoding one token through a feed-forward layer's first product.
        {"name": "act 1x8192x2048", "op": "act", "m": 1, "n": 8192, "k": 2048, "bias": True, "act": "silu",
         "residual": False, "pre": False, "out": "bf16"},
        # A short prompt through the second product, added to the stream that passes the layer by; ragged sizes.
        {"name": "act 200x4104x2056", "op": "act", "m": 200, "n": 4104, "k": 2056, "bias": True, "act": "none",
         "residual": True, "pre": False, "out": "f16"},
        # Prefill or training: activation and residual beside the tensor cores' work.
        {"name": "act 8192x8192x2048", "op": "act", "m": 8192, "n": 8192, "k": 2048, "bias": True, "act": "gelu",
         "residual": True, "pre": True, "out": "bf16"},
        # A small layer's training step.
        {"name": "act step 512x1024x1024", "op": "act step", "m": 512, "n": 1024, "k": 1024, "act": "gelu_tanh",
         "residual": False},
        # A large layer's training step.
        {"name": "act step 8192x4096x4096", "op": "act step", "m": 8192, "n": 4096, "k": 4096, "act": "silu",
         "residual": True},
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["experts", "experts", "experts", "step", "act", "act", "act step"])
    if op in ("experts", "step"):
        e = size(2, 64)
        c = {"op": op, "t": size(1, 8192), "top_k": min(e, rng.randint(1, 8)), "e": e, "n": size(64, 2048),
             "k": size(100, 4096), "pad": rng.choice([0, 0, size(1, 500)])}
        if op == "step":
            return {**c, "t": max(8, c["t"] // 2), "e": min(e, 16), "top_k": min(c["top_k"], 4, e, 16)}
        way = rng.choice(["forward", "dgrad", "wgrad"])
        if way == "wgrad":
            c = {**c, "t": max(1, c["t"] // 2), "e": min(e, 32), "top_k": min(c["top_k"], 4, e, 32)}
        return {**c, "way": way, "out": rng.choice(["bf16", "f16", "f32"])}
    c = {"op": op, "m": size(1, 8192), "n": size(64, 8192), "k": size(100, 2048),
         "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), "residual": rng.random() < 0.5}
    if op == "act step":
        return {**c, "m": max(16, c["m"]), "n": max(64, c["n"] // 2)}
    return {**c, "bias": rng.random() < 0.7, "pre": rng.random() < 0.3, "out": rng.choice(["bf16", "f16", "f32"])}


def work(case):
    blocks = lambda x: -(-x // BLOCK)  # noqa: E731
    if case["op"] in ("experts", "step"):
        t, e, n, k = case["t"] * case["top_k"], case["e"], case["n"], case["k"]
        used = e * (1 - (1 - case["top_k"] / e) ** case["t"])  # experts that some token chooses, for even routing
        if case["op"] == "step":
            # x, dy (16 bits), w (32 bits, of every expert) in; y, dx (16 bits), dw (32 bits) out
            return {"bytes": 4 * (t * k + t * n) + 8 * e * n * k, "flops": 6 * t * n * k}
        out = 4 if case["out"] == "f32" else 2
        if case["way"] == "wgrad":
            return {"bytes": int(t * (n + k) * (1 + 4 / BLOCK)) + e * n * k * out, "flops": 2 * t * n * k}
        b = t * k + 4 * t * blocks(k) + int(used * (n * k + 4 * blocks(n) * blocks(k))) + (t + case["pad"]) * n * out
        return {"bytes": b, "flops": 2 * t * n * k}
    m, n, k = case["m"], case["n"], case["k"]
    if case["op"] == "act":
        out = 4 if case["out"] == "f32" else 2
        b = m * k + n * k + 4 * m * blocks(k) + 4 * blocks(n) * blocks(k) + n * out
        return {"bytes": b + m * n * out * (1 + case["residual"] + case["pre"]), "flops": 2 * m * n * k}
    # x, dy, residual (16 bits), w (32 bits) in; y, dx, dw (16 bits) out; the values before the activation go out and in
    b = 2 * (2 * m * k + (2 + case["residual"] + 2 * (case["act"] != "none")) * m * n) + 6 * n * k
    return {"bytes": b, "flops": 6 * m * n * k}


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------


def spread(s, rows, cols, shape):
    """Scales repeated over their blocks of `rows` x `cols` entries, cut to `shape`."""
    return s.repeat_interleave(rows, -2).repeat_interleave(cols, -1)[..., : shape[-2], : shape[-1]]


def plain_quantize(x, rows, cols):
    """E4M3 values and scales of matrices with one scale for each block of rows x cols entries: s = amax / 448, and
    q = 448 x / amax rounded to the nearest E4M3 value (the factor split into 0.875 and 512, so that neither side
    overflows and the products of 16-bit entries are exact)."""
    x = x.float()
    m, k = x.shape[-2:]
    mb, kb = -(-m // rows), -(-k // cols)
    a = torch.nn.functional.pad(x.abs(), (0, kb * cols - k, 0, mb * rows - m))
    a = a.view(*x.shape[:-2], mb, rows, kb, cols).amax((-3, -1)).clamp_min(TINY)
    q = (x * 0.875) / spread(a * 2.0**-9, rows, cols, x.shape)
    return q.to(torch.float8_e4m3fn), a / E4M3_MAX


def plain_value(q, s, rows, cols):
    return q.float() * spread(s, rows, cols, q.shape)


def group_of(offsets, rows):
    """The group of every row, the number of groups for rows behind the last."""
    return torch.searchsorted(offsets[1:], torch.arange(rows, device=offsets.device, dtype=offsets.dtype), right=True)


def block_rows(offsets, rows):
    """The rows of x in the order of blocks of 128 that lie in one group each: group g's blocks start at offsets[g] //
    128 + g. Places without a row hold `rows`."""
    e = offsets.shape[0] - 1
    at = torch.arange(rows, device=offsets.device)
    g = group_of(offsets, rows)
    to = BLOCK * (offsets[g] // BLOCK + g) + at - offsets[g]
    places = (rows // BLOCK + e) * BLOCK
    src = torch.full((places + 1,), rows, dtype=torch.int64, device=offsets.device)
    src[torch.where(g < e, to, places)] = at
    return src[:places]


def with_zero(x):
    return torch.cat((x, x.new_zeros((1, x.shape[1]))))


def plain_quantize_columns(x, offsets):
    """x transposed, [K, 128 NB], in blocks of 128 rows of one group each."""
    x = with_zero(x.float())[block_rows(offsets, x.shape[0])]
    return plain_quantize(x.t(), 1, BLOCK)


def group_places(offsets, rows, cap):
    """Where each row goes in [E, cap] (all rows behind the last group to one place more)."""
    e = offsets.shape[0] - 1
    g = group_of(offsets, rows)
    return torch.where(g < e, g * cap + torch.arange(rows, device=offsets.device) - offsets[g], e * cap)


def by_group(x, places, e, cap):
    """[E, cap, K]: each group's rows, and zeros."""
    out = x.new_zeros((e * cap + 1, x.shape[1]))
    out[places] = x
    out[e * cap] = 0
    return out[: e * cap].view(e, cap, x.shape[1])


def plain_experts(x, w, offsets, cap):
    """x [T, K] times its group's w [E, K, N]: [T, N], rows behind the last group 0."""
    e = w.shape[0]
    places = group_places(offsets, x.shape[0], cap)
    y = torch.bmm(by_group(x, places, e, cap), w).view(e * cap, w.shape[2])
    return with_zero(y)[places]


def plain_experts_wgrad(a, b, offsets, cap):
    """a [M, 128 NB], b [N, 128 NB] in blocks of one group each: [E, M, N], the sums over each group's columns."""
    e = offsets.shape[0] - 1
    g = torch.arange(e, device=offsets.device)
    at = torch.arange(cap, device=offsets.device)
    cols = (BLOCK * (offsets[:-1] // BLOCK + g))[:, None] + at
    there = at < (offsets[1:] - offsets[:-1])[:, None]
    cols = cols.clamp_max(a.shape[1] - 1).view(-1)
    a = a[:, cols].view(a.shape[0], e, cap) * there
    b = b[:, cols].view(b.shape[0], e, cap) * there
    return torch.bmm(a.transpose(0, 1), b.permute(1, 2, 0))


def plain_step(x, w, dy, offsets, cap):
    qx, sx = plain_quantize(x, 1, BLOCK)
    qd, sd = plain_quantize(dy, 1, BLOCK)
    w8 = plain_value(*plain_quantize(w, BLOCK, BLOCK), BLOCK, BLOCK)
    y = plain_experts(plain_value(qx, sx, 1, BLOCK), w8.transpose(1, 2), offsets, cap)
    dx = plain_experts(plain_value(qd, sd, 1, BLOCK), w8, offsets, cap)
    dw = plain_experts_wgrad(plain_value(*plain_quantize_columns(dy, offsets), 1, BLOCK),
                             plain_value(*plain_quantize_columns(x, offsets), 1, BLOCK), offsets, cap)
    return y.to(x.dtype), dx.to(x.dtype), dw


def activate(x, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def activate_slope(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def plain_act(p, bias, act, residual, dtype):
    """(act(p + bias) + residual, p + bias), each rounded once."""
    if bias is not None:
        p = p + bias.float()
    y = activate(p, act)
    if residual is not None:
        y = y + residual.float()
    return y.to(dtype), p.to(dtype)


def plain_act_step(x, w, bias, act, residual, dy):
    w8 = plain_value(*plain_quantize(w, BLOCK, BLOCK), BLOCK, BLOCK)
    y, p = plain_act(plain_value(*plain_quantize(x, 1, BLOCK), 1, BLOCK) @ w8.t(), bias, act, residual, x.dtype)
    # the gradient before the activation, from what is kept of the forward pass: p in x's type
    d = dy.float() * activate_slope(p.float(), act)
    dx = plain_value(*plain_quantize(d, 1, BLOCK), 1, BLOCK) @ w8
    dw = plain_value(*plain_quantize(d.t(), 1, BLOCK), 1, BLOCK) @ \
        plain_value(*plain_quantize(x.float().t(), 1, BLOCK), 1, BLOCK).t()
    return y, dx.to(x.dtype), dw.to(x.dtype), d.sum(0).to(bias.dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def rows16(q):
    """The same matrix with rows that start on 16-byte boundaries, as quantised matrices are stored."""
    k = q.shape[-1]
    buf = torch.zeros((*q.shape[:-1], -(-k // 16) * 16), dtype=torch.uint8, device=q.device).view(q.dtype)
    buf[..., :k] = q
    return buf[..., :k]


def activations(g, m, k, dtype):
    """Normal entries, with some features much larger than the others, as hidden states have them."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn((1, k), generator=g, device="cuda"))
    return x.to(dtype)


def weights(g, *shape):
    return torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5


def expert_weights(g, e, n, k):
    """[E, N, K] E4M3 weights and their [E, ceil(N / 128), ceil(K / 128)] scales, a few experts at a time."""
    step = max(1, (1 << 28) // (n * k))
    q, s = zip(*(plain_quantize(weights(g, min(step, e - e0), n, k), BLOCK, BLOCK) for e0 in range(0, e, step)))
    return torch.cat([x.view(torch.uint8) for x in q]).view(torch.float8_e4m3fn), torch.cat(s)


def routing(g, t, top_k, e):
    """Where each expert's rows start, [E + 1], for tokens that choose top_k experts each, some experts oftener."""
    liking = torch.randn((t, e), generator=g, device="cuda") + 0.5 * torch.randn((1, e), generator=g, device="cuda")
    counts = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    chosen = liking.topk(top_k, 1).indices.flatten()
    counts.index_add_(0, chosen + 1, torch.ones_like(chosen))
    return counts.cumsum(0).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    if case["op"] in ("experts", "step"):
        e, n, k = case["e"], case["n"], case["k"]
        rows = case["t"] * case["top_k"] + case["pad"]
        st["offsets"] = routing(g, case["t"], case["top_k"], e)
        st["cap"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
        if case["op"] == "step":
            st["x"] = activations(g, rows, k, torch.bfloat16)
            st["w"] = weights(g, e, n, k)
            st["dy"] = activations(g, rows, n, torch.bfloat16) * 1e-3
        elif case["way"] == "wgrad":
            for name, width, size in (("a", n, 1e-3), ("b", k, 1.0)):
                q, st["s" + name] = plain_quantize_columns(activations(g, rows, width, torch.float32) * size,
                                                           st["offsets"])
                st[name] = rows16(q)
        else:
            q, st["sa"] = plain_quantize(activations(g, rows, k, torch.float32), 1, BLOCK)
            # forward: weights [E, N, K]; dgrad: [E, K, N], the contraction runs over their rows
            w, st["sb"] = expert_weights(g, e, *((n, k) if case["way"] == "forward" else (k, n)))
            st["a"], st["b"] = rows16(q), rows16(w)
    else:
        m, n, k = case["m"], case["n"], case["k"]
        dtype = DTYPES[case.get("out", "bf16")]
        has_bias = case.get("bias", True)
        st["bias"] = (0.1 * torch.randn(n, generator=g, device="cuda")).to(dtype) if has_bias else None
        st["residual"] = activations(g, m, n, dtype) if case["residual"] else None
        if case["op"] == "act":
            q, st["sa"] = plain_quantize(activations(g, m, k, torch.float32), 1, BLOCK)
            w, st["sb"] = plain_quantize(weights(g, n, k), BLOCK, BLOCK)
            st["a"], st["b"] = rows16(q), rows16(w)
        else:
            st["x"] = activations(g, m, k, dtype)
            st["w"] = weights(g, n, k)
            st["dy"] = activations(g, m, n, dtype) * 1e-3
    if own:
        import exact_modular_int8_gb300 as rg

        rg.library()
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(st):
    op = st["op"]
    if own:
        import exact_modular_int8_gb300 as rg

        if op == "experts" and st["way"] == "wgrad":
            return rg.grouped_wgrad_f8(st["a"], st["sa"], st["b"], st["sb"], st["offsets"],
                                       out_dtype=DTYPES[st["out"]], sync=False)
        if op == "experts":
            return rg.grouped_gemm_f8(st["a"], st["sa"], st["b"], st["sb"], st["offsets"],
                                      out_dtype=DTYPES[st["out"]], transb=st["way"] == "forward", sync=False)
        if op == "step":
            y, saved = rg.expert_linear_f8(st["x"], st["w"], st["offsets"], sync=False)
            dx, dw = rg.expert_linear_f8_backward(st["dy"], saved, sync=False)
            return y, dx, dw
        act = None if st["act"] == "none" else st["act"]
        if op == "act":
            return rg.scaled_gemm_act_f8(st["a"], st["sa"], st["b"], st["sb"], bias=st["bias"], act=act,
                                         residual=st["residual"], pre=st["pre"], out_dtype=DTYPES[st["out"]],
                                         sync=False)
        y, saved = rg.linear_act_f8(st["x"], st["w"], bias=st["bias"], act=act, residual=st["residual"], sync=False)
        dx, dw, db = rg.linear_act_f8_backward(st["dy"], saved, dw_dtype=torch.bfloat16, sync=False)
        return y, dx, dw, db
    if op == "step":
        return plain_step(st["x"], st["w"], st["dy"], st["offsets"], st["cap"])
    if op == "act step":
        return plain_act_step(*(st[x] for x in ("x", "w", "bias", "act", "residual", "dy")))
    a = plain_value(st["a"], st["sa"], 1, BLOCK)
    if op == "experts" and st["way"] == "wgrad":
        b = plain_value(st["b"], st["sb"], 1, BLOCK)
        return plain_experts_wgrad(a, b, st["offsets"], st["cap"]).to(DTYPES[st["out"]])
    b = plain_value(st["b"], st["sb"], BLOCK, BLOCK)
    if op == "experts":
        b = b.transpose(1, 2) if st["way"] == "forward" else b
        return plain_experts(a, b, st["offsets"], st["cap"]).to(DTYPES[st["out"]])
    y, p = plain_act(a @ b.t(), st["bias"], st["act"], st["residual"], DTYPES[st["out"]])
    return (y, p) if st["pre"] else y


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------


def exact_quantize(x, rows):
    """What the quantised matrix stands for, in 64 bits; rows = 1 or 128 rows to a block of 128 columns."""
    x = x.double()
    m = x.shape[0]
    out = torch.empty_like(x)
    for j in range(0, x.shape[1], BLOCK):
        part = x[:, j : j + BLOCK]
        top = part.abs().amax(1)
        if rows > 1:
            pad = torch.zeros(-(-m // rows) * rows, dtype=torch.float64, device=x.device)
            pad[:m] = top
            top = pad.view(-1, rows).amax(1).repeat_interleave(rows)[:m]
        top = top.clamp_min(TINY)[:, None]
        v = part * E4M3_MAX / top  # exact where it is a tie
        # E4M3: three stored significand bits, exponents from -6 up
        step = torch.exp2(torch.frexp(v)[1].clamp_min(-5).double() - 4)
        out[:, j : j + BLOCK] = torch.round(v / step) * step * (top / E4M3_MAX)
    return out


def exact_value(q, s, rows):
    """The same of given E4M3 values and scales."""
    out = q.double()
    for j in range(s.shape[1]):
        col = s[:, j].double().repeat_interleave(rows)[: q.shape[0]]
        out[:, j * BLOCK : (j + 1) * BLOCK] *= col[:, None]
    return out


def exact_act(x, act):
    """(the activation, its slope) in 64 bits."""
    x = x.double()
    if act == "relu":
        return x.clamp_min(0), (x > 0).double()
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * (1 - s)
    if act == "gelu":
        c = torch.special.ndtr(x)
        return x * c, c + x * torch.exp(-x * x / 2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        # (1 + tanh(u)) / 2 = sigmoid(2 u)
        s = torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (x + 0.044715 * x**3))
        return x * s, s + x * s * (1 - s) * 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * x**2)
    return x, torch.ones_like(x)


def exact(case, seed):
    st = prepare(case, seed)
    op, n, k = case["op"], case["n"], case["k"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if op in ("experts", "step"):
        off = st["offsets"].tolist()
        rows = case["t"] * case["top_k"] + case["pad"]
        if op == "experts" and case["way"] == "wgrad":
            a, b = exact_value(st["a"], st["sa"], 1), exact_value(st["b"], st["sb"], 1)
            out = torch.zeros((case["e"], n, k), **f64)
            for g in range(case["e"]):
                at = slice(BLOCK * (off[g] // BLOCK + g), BLOCK * (off[g] // BLOCK + g) + off[g + 1] - off[g])
                out[g] = a[:, at] @ b[:, at].t()
            return out
        if op == "experts":
            a, out = exact_value(st["a"], st["sa"], 1), torch.zeros((rows, n), **f64)
            for g in range(case["e"]):
                at = slice(off[g], off[g + 1])
                b = exact_value(st["b"][g], st["sb"][g], BLOCK)
                out[at] = a[at] @ (b.t() if case["way"] == "forward" else b)
            return out
        x, dy = exact_quantize(st["x"], 1), exact_quantize(st["dy"], 1)
        y, dx, dw = torch.zeros((rows, n), **f64), torch.zeros((rows, k), **f64), torch.zeros((case["e"], n, k), **f64)
        for g in range(case["e"]):
            at = slice(off[g], off[g + 1])
            w = exact_quantize(st["w"][g], BLOCK)
            y[at], dx[at] = x[at] @ w.t(), dy[at] @ w
            if off[g + 1] > off[g]:
                dw[g] = exact_quantize(st["dy"][at].t(), 1) @ exact_quantize(st["x"][at].t(), 1).t()
        return y, dx, dw
    bias = 0 if st["bias"] is None else st["bias"].double()
    residual = 0 if st["residual"] is None else st["residual"].double()
    if op == "act":
        p = exact_value(st["a"], st["sa"], 1) @ exact_value(st["b"], st["sb"], BLOCK).t() + bias
        y = exact_act(p, case["act"])[0] + residual
        return (y, p) if case["pre"] else y
    w = exact_quantize(st["w"], BLOCK)
    p = exact_quantize(st["x"], 1) @ w.t() + bias
    d = st["dy"].double() * exact_act(p.to(st["x"].dtype), case["act"])[1]
    dw = exact_quantize(d.t(), 1) @ exact_quantize(st["x"].t(), 1).t()
    return exact_act(p, case["act"])[0] + residual, exact_quantize(d, 1) @ w, dw, d.sum(0)
