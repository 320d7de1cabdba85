"""Cases of the layer norm, of 4-bit floating point with its linear layer, and of orthogonalised updates.

Five operators:

  norm           y = (x - mean) / sqrt(var + eps) gamma + beta over each row; with its backward pass dx, dgamma and dbeta too
  fp4            a matrix in 4-bit floating point, blocks of 1 x 32, and the values read back
  fp4_linear     y = Q(x) W^T + bias for a weight kept in 4 bits: x is quantized within the call
  orthogonalize  five Newton-Schulz steps on a matrix scaled to norm 1: X <- a X + (b A + c A A) X with A = X X^T
  muon           one step over a list of matrices: momentum, its orthogonalised update, decoupled weight decay

Q: a block's scale is 2^e with the smallest e >= -127 for which no magnitude exceeds 6 * 2^e; values are rounded to the nearest
e2m1 multiple of it (0, 0.5, 1, 1.5, 2, 3, 4, 6), ties to the even code.
"""

import torch

own = False

D_350M, FFN_350M, CONTEXT_350M, LAYERS_350M = 1024, 4096, 1024, 24
D_7B, FFN_7B = 4096, 11008
TOKENS_7B = 4 * 4096

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}

EPS = 1e-5
NS_STEPS, NS_EPS, NS_A, NS_B, NS_C = 5, 1e-7, 3.4445, -4.7750, 2.0315
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01


def listed():
    return [
        # one decoded token before a 7B-shaped projection: latency
        {"name": "norm_1_token", "op": "norm", "rows": 1, "width": D_7B, "type": "bf16", "gtype": "bf16", "backward": False},
        # fp32 activations of a small model, ragged in both sizes, in training
        {"name": "norm_ragged", "op": "norm", "rows": 1111, "width": 1003, "type": "fp32", "gtype": "fp32", "backward": True},
        # a pre-norm of the 7B set over four sequences of 4,096 tokens in training, its vectors in 32 bits
        {"name": "norm_7b", "op": "norm", "rows": TOKENS_7B, "width": D_7B, "type": "bf16", "gtype": "fp32", "backward": True},
        # a small fp32 matrix whose rows end inside a block
        {"name": "fp4_ragged", "op": "fp4", "rows": 777, "width": 1003, "type": "fp32"},
        # one feed-forward matrix of the 7B set, quantized for serving
        {"name": "fp4_weight", "op": "fp4", "rows": FFN_7B, "width": D_7B, "type": "bf16"},
        # one token through a 7B-shaped projection: latency, and reading the weight once
        {"name": "fp4_1_token", "op": "fp4_linear", "tokens": 1, "inputs": D_7B, "outputs": D_7B, "type": "bf16", "bias": False},
        # a ragged prompt through a layer whose sizes are no multiple of anything, with a bias
        {"name": "fp4_linear_ragged", "op": "fp4_linear", "tokens": 257, "inputs": 1003, "outputs": 2051, "type": "fp16", "bias": True},
        # a prompt batch of four times 4,096 tokens
        {"name": "fp4_prompt", "op": "fp4_linear", "tokens": TOKENS_7B, "inputs": D_7B, "outputs": FFN_7B, "type": "bf16", "bias": False},
        # one small fp32 update of odd sizes, taller than wide: latency
        {"name": "orthogonalize_ragged", "op": "orthogonalize", "rows": 777, "width": 301, "type": "fp32"},
        # the update of one feed-forward matrix of the 7B set
        {"name": "orthogonalize_7b", "op": "orthogonalize", "rows": FFN_7B, "width": D_7B, "type": "bf16"},
        # a few small matrices of different shapes, one without a gradient so far
        {"name": "muon_small", "op": "muon", "set": "small", "type": "fp32", "gtype": "fp32"},
        # the square and the feed-forward matrices of the 350M set
        {"name": "muon_350m", "op": "muon", "set": "350m", "type": "fp32", "gtype": "bf16"},
    ]


def log_uniform(rng, low, high):
    return min(high, int(low * (high / low) ** rng.random() + 0.5))


def draw(rng):
    op = rng.choice(["norm", "norm", "fp4", "fp4_linear", "fp4_linear", "orthogonalize", "orthogonalize", "muon"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "fp4"):
        width = log_uniform(rng, 32, FFN_7B)
        if rng.random() < 0.5:  # sizes of real layers are mostly multiples of 64
            width = -(-width // 64) * 64
        most = (TOKENS_7B if op == "norm" else FFN_7B) * D_7B
        rows = log_uniform(rng, 1, min(TOKENS_7B, most // (width * BYTES[dtype] // 2)))
        case = {"op": op, "rows": rows, "width": width, "type": dtype}
        if op == "norm":
            case.update(gtype=rng.choice([dtype, "fp32"]), backward=rng.random() < 0.7)
        return case
    if op == "fp4_linear":
        inputs, outputs = log_uniform(rng, 64, FFN_7B), log_uniform(rng, 64, FFN_7B)
        if rng.random() < 0.5:
            inputs, outputs = -(-inputs // 64) * 64, -(-outputs // 64) * 64
        tokens = log_uniform(rng, 1, TOKENS_7B)
        tokens = max(1, min(tokens, TOKENS_7B * D_7B * FFN_7B // (inputs * outputs)))
        if dtype == "fp32":
            tokens = max(1, tokens // 2)
        return {"op": op, "tokens": tokens, "inputs": inputs, "outputs": outputs, "type": dtype, "bias": rng.random() < 0.5}
    if op == "orthogonalize":
        small = log_uniform(rng, 16, 2048)
        large = log_uniform(rng, small, 8 * small if small > 500 else 4096)
        if rng.random() < 0.5:
            small, large = -(-small // 64) * 64, -(-large // 64) * 64
        if rng.random() < 0.5:
            small, large = large, small
        return {"op": op, "rows": small, "width": large, "type": dtype}
    shapes = [[log_uniform(rng, 16, 1500), log_uniform(rng, 16, 1500)] for _ in range(rng.randrange(1, 4))]
    copies = rng.randrange(1, 7)
    return {"op": op, "set": "drawn", "shapes": ";".join(f"{r}x{c}" for r, c in shapes for _ in range(copies)), "type": dtype,
            "gtype": rng.choice([dtype, "fp32"]) if dtype == "fp32" else dtype}


def shapes_of(case):
    """(rows, columns) of a muon case's matrices."""
    if case["set"] == "small":
        return [(300, 200), (200, 300), (64, 1000), (64, 1000), (500, 17)]
    if case["set"] == "drawn":
        return [tuple(int(n) for n in s.split("x")) for s in case["shapes"].split(";")]
    d, ffn = D_350M, FFN_350M
    return [(d, d), (ffn, d), (d, ffn)] * LAYERS_350M


def normal(shape, std, g, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def activations(rows, width, g, dtype):
    """N(0, 1) with a few channels thirty times as large, every row of its own size and offset, and the last rows zero, as padding is."""
    x = torch.randn((rows, width), generator=g, device="cuda")
    loud = torch.rand(width, generator=g, device="cuda") < 0.005
    x = torch.where(loud, 30.0 * x, x)
    x = x * torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda")) + 0.3 * torch.randn((rows, 1), generator=g, device="cuda")
    if rows > 16:
        x[rows - rows // 16:] = 0.0
    return x.to(dtype)


def update(rows, cols, g, dtype=torch.float32):
    """What a weight's gradient looks like: a few strong directions (the inputs' and outputs' common ones) over many weak ones."""
    rank = max(1, min(rows, cols, 64) // 4)
    size = torch.exp(-3.0 * torch.arange(rank, device="cuda") / rank)
    strong = (torch.randn((rows, rank), generator=g, device="cuda") * size) @ torch.randn((rank, cols), generator=g, device="cuda")
    return (1e-3 * (strong + torch.randn((rows, cols), generator=g, device="cuda"))).to(dtype)


def flat(matrices):
    """One buffer that holds them all, and the list of its views."""
    buffer = torch.cat([m.reshape(-1) for m in matrices])
    parts = buffer.split([m.numel() for m in matrices])
    return buffer, [part.view(m.shape) for part, m in zip(parts, matrices)]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    dtype = TYPES[case["type"]]
    if op == "norm":
        t, d, vectors = case["rows"], case["width"], TYPES[case["gtype"]]
        s["x"] = activations(t, d, g, dtype)
        s["gamma"], s["beta"] = 1.0 + normal((d,), 0.2, g), normal((d,), 0.1, g)
        s["gamma"], s["beta"] = s["gamma"].to(vectors), s["beta"].to(vectors)
        if case["backward"]:
            s["dy"] = normal((t, d), 1e-3, g, dtype)
    elif op == "fp4":
        s["x"] = normal((case["rows"], case["width"]), 0.02, g, dtype)
        s["x"][:, ::61] *= 20  # columns with outliers
    elif op == "fp4_linear":
        t, k, n = case["tokens"], case["inputs"], case["outputs"]
        s["x"] = activations(t, k, g, dtype)
        s["bias"] = normal((n,), 0.1, g, dtype) if case["bias"] else None
        w = normal((n, k), 0.02, g, dtype)
        if own:
            from block_wise_dynamic_gb300 import fp4

            s["w"] = fp4.quantize(w)
        else:
            s["w"] = quantize(w)
    elif op == "orthogonalize":
        s["g"] = update(case["rows"], case["width"], g, dtype)
    else:
        shapes, gtype = shapes_of(case), TYPES[case["gtype"]]
        s["p"], s["list_p"] = flat([normal(shape, 0.02, g, dtype) for shape in shapes])
        s["list_g"] = [update(*shape, g, gtype) for shape in shapes]
        s["m"], s["list_m"] = flat([5.0 * update(*shape, g) for shape in shapes])
        if len(shapes) > 1:  # a matrix that nothing has reached so far
            s["list_g"][-1].zero_()
            s["list_m"][-1].zero_()
        if own:
            from block_wise_dynamic_gb300 import muon

            s["args"] = muon.MuonArgs(s["list_p"], s["list_g"], s["list_m"])
    return s


# plain forms


def quantize(x):
    """Magnitudes' codes (0 to 7, the sign at 8) of x and each block's exponent byte (e + 127)."""
    r, c = x.shape
    blocks = torch.zeros((r, -(-c // 32) * 32), device=x.device)
    blocks[:, :c] = x
    blocks = blocks.view(r, -1, 32)
    largest = blocks.abs().amax(2, keepdim=True)
    # 6 = 1.5 * 2^2: the exponent field, one more where the fraction is over 0.5, less two
    byte = (((largest.view(torch.int32) + 0x3FFFFF) >> 23) - 2).clamp(min=0)
    v = blocks * ((254 - byte) << 23).view(torch.float32)
    a = v.abs()
    code = torch.where(a <= 0.25, 0, 1)
    # a tie goes to the even code: up from an odd one
    code = code + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return (code + 8 * (blocks < 0)).to(torch.uint8), byte, c


def values(codes, byte, c):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    v = torch.cat([grid, -grid])[codes.long()]
    scale = torch.where(byte > 0, byte << 23, 1 << 22).to(torch.int32).view(torch.float32)
    return (v * scale).reshape(v.shape[0], -1)[:, :c]


def plain_norm(s):
    x, gamma, dtype = s["x"].float(), s["gamma"].float(), s["x"].dtype
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
    xh = (x - mean) * rstd
    y = (xh * gamma + s["beta"].float()).to(dtype)
    if not s["case"]["backward"]:
        return y
    dy = s["dy"].float()
    h = dy * gamma
    dx = rstd * (h - h.mean(1, keepdim=True) - xh * (h * xh).mean(1, keepdim=True))
    return [y, dx.to(dtype), (dy * xh).sum(0).to(s["gamma"].dtype), dy.sum(0).to(s["gamma"].dtype)]


def plain_linear(s):
    y = values(*quantize(s["x"])) @ values(*s["w"]).t()
    return (y if s["bias"] is None else y + s["bias"].float()).to(s["x"].dtype)


def newton_schulz(g):
    x = g.float()
    if x.shape[0] > x.shape[1]:
        return newton_schulz(x.t()).t()
    x = x / (x.square().sum().sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        a = x @ x.t()
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x


def plain_muon(s):
    for p, g, m in zip(s["list_p"], s["list_g"], s["list_m"]):
        m.mul_(MOMENTUM).add_(g.float())
        o = newton_schulz(g.float() + MOMENTUM * m)
        p.copy_(p.float() * (1 - LR * DECAY) - (LR * 0.2 * max(p.shape) ** 0.5) * o)
    return [s["p"], s["m"]]


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "norm":
            return plain_norm(s)
        if op == "fp4":
            return values(*quantize(s["x"])).to(s["x"].dtype)
        if op == "fp4_linear":
            return plain_linear(s)
        return newton_schulz(s["g"]).to(s["g"].dtype).contiguous() if op == "orthogonalize" else plain_muon(s)
    from block_wise_dynamic_gb300 import fp4, muon, norm

    if op == "norm":
        if not s["case"]["backward"]:
            return norm.forward(s["x"], s["gamma"], s["beta"], EPS, need_stats=False)[0]
        y, mean, rstd = norm.forward(s["x"], s["gamma"], s["beta"], EPS)
        return [y, *norm.backward(s["dy"], s["x"], s["gamma"], mean, rstd)]
    if op == "fp4":
        return fp4.quantize(s["x"]).dequantize()
    if op == "fp4_linear":
        return fp4.linear(s["x"], s["w"], s["bias"])
    if op == "orthogonalize":
        return muon.orthogonalize(s["g"])
    s["args"].step(lr=LR, momentum=MOMENTUM, weight_decay=DECAY)
    return [s["p"], s["m"]]


def newton_schulz_flops(rows, cols):
    m, n = min(rows, cols), max(rows, cols)
    # A and A A are symmetric: half of each
    return NS_STEPS * (m * m * n + m ** 3 + 2 * m * m * n)


def work(case):
    op, b = case["op"], BYTES[case["type"]]
    if op == "norm":
        n, d = case["rows"] * case["width"], case["width"] * BYTES[case["gtype"]]
        if not case["backward"]:
            return {"bytes": 2 * b * n + 2 * d, "flops": 8 * n}
        return {"bytes": 4 * b * n + 4 * d, "flops": 22 * n}
    if op == "fp4":
        n = case["rows"] * case["width"]
        return {"bytes": 2 * b * n, "flops": 4 * n}
    if op == "fp4_linear":
        t, k, n = case["tokens"], case["inputs"], case["outputs"]
        return {"bytes": b * t * (k + n) + n * (-(-k // 2) + -(-k // 32)) + (b * n if case["bias"] else 0), "flops": 2 * t * k * n}
    if op == "orthogonalize":
        return {"bytes": 2 * b * case["rows"] * case["width"], "flops": newton_schulz_flops(case["rows"], case["width"])}
    shapes = shapes_of(case)
    n = sum(r * c for r, c in shapes)
    return {"bytes": (2 * b + BYTES[case["gtype"]] + 8) * n, "flops": sum(newton_schulz_flops(r, c) + 8 * r * c for r, c in shapes)}


# the definitions in 64 bits


def power_of_two(e):
    """2^e in 64 bits, exactly: its exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def exact_q(x):
    x = x.double()
    rows, cols = x.shape
    v = torch.nn.functional.pad(x, (0, -cols % 32))
    top = v.reshape(rows, -1, 32).abs().amax(2)
    half, power = torch.frexp(top / 6.0)  # top / 6 = half * 2^power with half in [0.5, 1)
    e = torch.where(half == 0.5, power - 1, power).clamp(min=-127)
    e = torch.where(top == 0, torch.zeros_like(e), e).repeat_interleave(32, 1)
    q = v * power_of_two(-e)
    grain = power_of_two((torch.frexp(q)[1] - 1).clamp(min=0) - 1)  # one fraction bit; 1 is the least normal
    return ((q / grain).round() * grain * power_of_two(e))[:, :cols]


def exact_orthogonal(g):
    # the polynomial acts on the singular values of the normalised matrix; here by products on the shorter side
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x / (torch.linalg.matrix_norm(x) + NS_EPS)
    gram = x.t() @ x if tall else x @ x.t()
    total = torch.eye(gram.shape[0], dtype=torch.float64, device=g.device)
    for _ in range(NS_STEPS):
        # all powers of one symmetric matrix commute: X_k = total_k X_0, A_k = total_k^2 A_0
        a = total @ gram @ total
        total = NS_A * total + (NS_B * a + NS_C * a @ a) @ total
        total = 0.5 * (total + total.t())
    return x @ total if tall else total @ x


def exact(case, seed):
    global own
    was, own = own, False
    try:
        # the linear layer's weight before it is quantized: made as prepare makes it
        s = prepare(case, seed)
        if case["op"] == "fp4_linear":
            w = weight(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "norm":
        x, gamma, beta = s["x"].double(), s["gamma"].double(), s["beta"].double()
        centred = x - x.mean(1, keepdim=True)
        scale = 1.0 / torch.sqrt((centred ** 2).mean(1, keepdim=True) + EPS)
        y = centred * scale * gamma + beta
        if not case["backward"]:
            return y
        dy = s["dy"].double()
        h = dy * gamma
        along = (h * centred).mean(1, keepdim=True) * scale ** 2
        dx = scale * (h - h.mean(1, keepdim=True) - centred * along)
        return [y, dx, (dy * centred * scale).sum(0), dy.sum(0)]
    if op == "fp4":
        return exact_q(s["x"])
    if op == "fp4_linear":
        y = exact_q(s["x"]) @ exact_q(w).t()
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "orthogonalize":
        return exact_orthogonal(s["g"])
    ps, ms = [], []
    for p, g, m in zip(s["list_p"], s["list_g"], s["list_m"]):
        g, m = g.double(), 0.95 * m.double() + g.double()
        ms.append(m)
        ps.append(p.double() * (1 - 0.02 * 0.01) - 0.02 * 0.2 * max(p.shape) ** 0.5 * exact_orthogonal(g + 0.95 * m))
    return [flat(ps)[0], flat(ms)[0]]


def weight(case, seed):
    """The weight that prepare quantizes for this case and seed."""
    g = torch.Generator("cuda").manual_seed(seed)
    dtype, t, k, n = TYPES[case["type"]], case["tokens"], case["inputs"], case["outputs"]
    activations(t, k, g, dtype)
    if case["bias"]:
        normal((n,), 0.1, g, dtype)
    return normal((n, k), 0.02, g, dtype)
