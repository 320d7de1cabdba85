"""Cases of the 8-bit floating point linear layer, of the AdamW step with 32-bit states and of the global gradient norm.

Four operators:

  linear  y = Q(x) W^T + bias for a weight kept in 8 bits: x is quantized in blocks of 1 x 128 within the call
  train   a linear layer's forward and backward pass: the weight (blocks of 128 x 128), x and dy (blocks of 1 x 128 and of
          128 x 1, each along the axis that its product sums over) are quantized within the call; gives y, dx, dw, dbias
  adamw   one AdamW step over a list of tensors with both moments in fp32, the gradients times a factor held on the device
  norm    the 2-norm of a list of gradients and the factor that clips it

Q: a block's scale is 2^e with the smallest e >= -127 for which no magnitude exceeds 448 * 2^e; values are rounded to the nearest
e4m3 multiple of it, ties to even.
"""

import torch

own = False

D_350M, FFN_350M, VOCAB_350M, CONTEXT_350M, LAYERS_350M = 1024, 4096, 50304, 1024, 24
D_7B, FFN_7B, VOCAB_7B = 4096, 11008, 32000

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}

LR, BETA1, BETA2, EPS, DECAY, MAX_NORM = 1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0


def listed():
    return [
        # one token through a 7B-shaped projection: latency, and reading the weight once
        {"name": "linear_1_token", "op": "linear", "tokens": 1, "inputs": D_7B, "outputs": D_7B, "type": "bf16", "bias": False},
        # a small batch of sequences decoded together, into the feed-forward width
        {"name": "linear_33_tokens", "op": "linear", "tokens": 33, "inputs": D_7B, "outputs": FFN_7B, "type": "bf16", "bias": False},
        # a ragged prompt through a layer whose sizes are no multiple of anything, with a bias
        {"name": "linear_ragged", "op": "linear", "tokens": 777, "inputs": 1003, "outputs": 2051, "type": "fp16", "bias": True},
        # a prompt batch of four times 4,096 tokens
        {"name": "linear_prompt", "op": "linear", "tokens": 16384, "inputs": D_7B, "outputs": FFN_7B, "type": "bf16", "bias": False},
        # one feed-forward matrix of the 350M set in training, with its bias
        {"name": "train_350m", "op": "train", "tokens": 4 * CONTEXT_350M, "inputs": D_350M, "outputs": FFN_350M, "type": "bf16", "bias": True},
        # fp32 activations (as the stable embedding layer gives them), ragged in every size
        {"name": "train_ragged_fp32", "op": "train", "tokens": 1111, "inputs": 1003, "outputs": 517, "type": "fp32", "bias": True},
        # one feed-forward matrix of the 7B set over two sequences of 4,096 tokens
        {"name": "train_7b", "op": "train", "tokens": 8192, "inputs": D_7B, "outputs": FFN_7B, "type": "bf16", "bias": False},
        # the norms and biases of the 350M set, which stay in 32 bits beside 8-bit matrices: launch latency
        {"name": "adamw_vectors", "op": "adamw", "set": "vectors", "type": "fp32", "gtype": "fp32", "clip": False},
        # the whole 350M set with 32-bit states, its gradients clipped
        {"name": "adamw_350m", "op": "adamw", "set": "all", "type": "fp32", "gtype": "bf16", "clip": True},
        # the 7B set's token embedding in 32 bits, bf16 parameters
        {"name": "adamw_embedding", "op": "adamw", "set": "embedding", "type": "bf16", "gtype": "bf16", "clip": False},
        # the norm of a few small gradients: latency
        {"name": "norm_vectors", "op": "norm", "set": "vectors", "gtype": "fp32"},
        # the norm over all gradients of the 350M set
        {"name": "norm_350m", "op": "norm", "set": "all", "gtype": "bf16"},
    ]


def log_uniform(rng, low, high):
    return min(high, int(low * (high / low) ** rng.random() + 0.5))


def draw(rng):
    op = rng.choice(["linear", "linear", "train", "train", "adamw", "norm"])
    types = ["bf16", "bf16", "fp16", "fp32"]
    if op in ("linear", "train"):
        tokens = log_uniform(rng, 1, 16384 if op == "linear" else 8192)
        inputs, outputs = log_uniform(rng, 64, FFN_7B), log_uniform(rng, 64, FFN_7B)
        if rng.random() < 0.5:  # sizes of real layers are mostly multiples of 64
            inputs, outputs = -(-inputs // 64) * 64, -(-outputs // 64) * 64
        inputs, outputs = min(inputs, FFN_7B), min(outputs, FFN_7B)
        tokens = max(1, min(tokens, (16384 if op == "linear" else 8192) * D_7B * FFN_7B // (inputs * outputs)))
        return {"op": op, "tokens": tokens, "inputs": inputs, "outputs": outputs, "type": rng.choice(types), "bias": rng.random() < 0.5}
    case = {"op": op, "set": "drawn", "tensors": log_uniform(rng, 1, 400), "elements": log_uniform(rng, 1000, 200_000_000),
            "sizes": rng.randrange(1 << 30), "align": rng.choice([1, 2, 8, 64]), "gtype": rng.choice(types)}
    if op == "adamw":
        case.update(type=rng.choice(types), clip=rng.random() < 0.5)
        if case["type"] != "fp32" and case["gtype"] == "fp32":
            case["gtype"] = case["type"]
    return case


def tensor_sizes(case):
    """The list's tensor sizes, and how many elements each one's start is rounded up to."""
    if case["set"] == "embedding":
        return [VOCAB_7B * D_7B], 64
    if case["set"] == "drawn":
        g = torch.Generator().manual_seed(case["sizes"])
        share = torch.exp(4.0 * torch.rand(case["tensors"], generator=g, dtype=torch.float64))
        return [max(1, int(case["elements"] * float(s))) for s in share / share.sum()], case["align"]
    d, ffn = D_350M, FFN_350M
    vectors = [d, d, 3 * d, d, d, d, ffn, d] * LAYERS_350M + [d, d]
    if case["set"] == "vectors":
        return vectors, 64
    return [VOCAB_350M * d, CONTEXT_350M * d] + vectors + [3 * d * d, d * d, d * ffn, ffn * d] * LAYERS_350M, 64


def places(case):
    """[(offset, size)] of the list's tensors in one flat buffer, and the buffer's size."""
    sizes, align = tensor_sizes(case)
    at, end = [], 0
    for n in sizes:
        end = -(-end // align) * align
        at.append((end, n))
        end += n
    return at, end


def normal(shape, std, g, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def activations(tokens, width, g, dtype):
    """N(0, 1) with a few channels thirty times as large, and the last tokens zero, as padding is."""
    x = torch.randn((tokens, width), generator=g, device="cuda")
    loud = torch.rand(width, generator=g, device="cuda") < 0.005
    x = torch.where(loud, 30.0 * x, x)
    if tokens > 16:
        x[tokens - tokens // 16:] = 0.0
    return x.to(dtype)


def gradients(tokens, width, g, dtype):
    """N(0, 1e-3), each token's gradient of its own size, and the last tokens' zero."""
    dy = torch.randn((tokens, width), generator=g, device="cuda")
    dy *= 1e-3 * torch.exp(torch.randn((tokens, 1), generator=g, device="cuda"))
    if tokens > 16:
        dy[tokens - tokens // 16:] = 0.0
    return dy.to(dtype)


def flat_lists(case, seed):
    """The tensors of adamw and norm: flat buffers and the list's views of them; elements between tensors stay zero."""
    g = torch.Generator("cuda").manual_seed(seed)
    at, n = places(case)
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    for start, size in at:
        used[start:start + size] = True
    s = {"case": case}

    def buffer(name, values):
        s[name] = torch.where(used, values, torch.zeros((), dtype=values.dtype, device="cuda"))

    buffer("g", normal(n, 1e-3, g, TYPES[case["gtype"]]))
    names = ["g"]
    if case["op"] == "adamw":
        names = ["p", "g", "m", "v"]
        buffer("p", normal(n, 0.02, g, TYPES[case["type"]]))
        buffer("m", normal(n, 3e-4, g))
        buffer("v", normal(n, 1e-3, g).square())
    for name in names:
        s["list_" + name] = [s[name][start:start + size] for start, size in at]
    return s


def prepare(case, seed):
    if case["op"] in ("adamw", "norm"):
        s = flat_lists(case, seed)
        if case["op"] == "adamw":
            s["step"] = 100  # steps taken so far
            s["scale"] = torch.full((1,), 0.37, device="cuda")  # an earlier call's factor
        if own:
            import block_wise_dynamic_gb300 as bwd

            if case["op"] == "norm" or case["clip"]:
                s["norm"] = bwd.GradNorm(s["list_g"])
            if case["op"] == "adamw":
                s["args"] = bwd.MultiTensorArgs32(s["list_p"], s["list_g"], s["list_m"], s["list_v"])
        return s
    g = torch.Generator("cuda").manual_seed(seed)
    dtype, t, k, n = TYPES[case["type"]], case["tokens"], case["inputs"], case["outputs"]
    s = {"case": case, "x": activations(t, k, g, dtype), "bias": normal((n,), 0.1, g, dtype) if case["bias"] else None}
    w = normal((n, k), 0.02, g, dtype)
    if case["op"] == "train":
        s["w"], s["dy"] = w, gradients(t, n, g, dtype)
    elif own:
        from block_wise_dynamic_gb300 import fp8

        s["w"] = fp8.quantize(w, "tiles")
    else:
        s["w"] = quantize(w, 128, 128)
    return s


# plain forms


def quantize(x, rows, cols):
    """e4m3 codes of x and the exponent byte (e + 127) of each block of rows x cols."""
    r, c = x.shape
    br, bc = -(-r // rows), -(-c // cols)
    padded = torch.zeros((br * rows, bc * cols), device=x.device)
    padded[:r, :c] = x
    blocks = padded.view(br, rows, bc, cols)
    largest = blocks.abs().amax((1, 3), keepdim=True)
    # 448 = 1.75 * 2^8: the exponent field, one more where the fraction is over 0.75, less eight
    byte = (((largest.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=0)
    codes = (blocks * ((254 - byte) << 23).view(torch.float32)).to(torch.float8_e4m3fn)
    return codes, byte, r, c


def values(codes, byte, r, c):
    scale = torch.where(byte > 0, byte << 23, 1 << 22).to(torch.int32).view(torch.float32)
    v = codes.to(torch.float32) * scale
    return v.reshape(v.shape[0] * v.shape[1], -1)[:r, :c]


def plain_linear(s):
    x, dtype = s["x"], s["x"].dtype
    y = values(*quantize(x, 1, 128)) @ values(*s["w"]).t()
    return (y if s["bias"] is None else y + s["bias"].float()).to(dtype)


def plain_train(s):
    x, dy, dtype = s["x"], s["dy"], s["x"].dtype
    w = values(*quantize(s["w"], 128, 128))
    y = values(*quantize(x, 1, 128)) @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    dx = values(*quantize(dy, 1, 128)) @ w
    dw = values(*quantize(dy, 128, 1)).t() @ values(*quantize(x, 128, 1))
    db = None if s["bias"] is None else dy.float().sum(0).to(dtype)
    return [y.to(dtype), dx.to(dtype), dw.to(dtype), db]


def plain_norm(s):
    norm = s["g"].float().square().sum().sqrt()
    return [torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0), norm]


def plain_adamw(s):
    scale = plain_norm(s)[0] if s["case"]["clip"] else s["scale"]
    p, m, v = s["p"], s["m"], s["v"]
    s["step"] += 1
    bc1, bc2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    g = s["g"].float() * scale
    m.mul_(BETA1).add_(g * (1 - BETA1))
    v.mul_(BETA2).add_(g * g * (1 - BETA2))
    update = m / (v.sqrt() / bc2 ** 0.5 + EPS)
    p.copy_(p.float() * (1 - LR * DECAY) - update * (LR / bc1))
    return [p, m, v]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"linear": plain_linear, "train": plain_train, "norm": plain_norm, "adamw": plain_adamw}[op](s)
    from block_wise_dynamic_gb300 import fp8

    if op == "linear":
        return fp8.linear(s["x"], s["w"], s["bias"])
    if op == "train":
        w = fp8.quantize(s["w"], "tiles")
        y, xq = fp8.forward(s["x"], w, s["bias"])
        dx, dw, db = fp8.backward(s["dy"], xq, w, need_bias=s["bias"] is not None)
        return [y, dx, dw, db]
    if op == "norm":
        scale, norm = s["norm"].clip_scale(MAX_NORM)
        return [scale.view(()), norm.view(())]
    scale = s["norm"].clip_scale(MAX_NORM)[0] if s["case"]["clip"] else s["scale"]
    s["step"] += 1
    s["args"].step(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, step=s["step"], grad_scale=scale)
    return [s["p"], s["m"], s["v"]]


def work(case):
    if case["op"] in ("adamw", "norm"):
        n = sum(tensor_sizes(case)[0])
        read = BYTES[case["gtype"]] * n
        if case["op"] == "norm":
            return {"bytes": read + 8, "flops": 2 * n}
        return {"bytes": read + (16 + 2 * BYTES[case["type"]]) * n, "flops": (14 + 2 * case["clip"]) * n}
    t, k, n, b = case["tokens"], case["inputs"], case["outputs"], BYTES[case["type"]]
    bias = b * n if case["bias"] else 0
    if case["op"] == "linear":
        return {"bytes": b * t * (k + n) + n * k + -(-n // 128) * -(-k // 128) + bias, "flops": 2 * t * k * n}
    return {"bytes": b * (2 * t * k + 2 * t * n + 2 * n * k) + 2 * bias, "flops": 6 * t * k * n}


# the definitions in 64 bits


def exact_q(x, axis):
    """What x stands for after quantization: axis 0 or 1, blocks of 128 along it; None, blocks of 128 x 128."""
    x = x.double()
    v = x
    for a in (0, 1):
        if axis in (None, a):
            pad = [0, 0, 0, 0]
            pad[3 - 2 * a] = -v.shape[a] % 128
            v = torch.nn.functional.pad(v, pad)
    rows, cols = v.shape
    if axis == 1:
        top = v.reshape(rows, -1, 128).abs().amax(2).repeat_interleave(128, 1)
    elif axis == 0:
        top = v.reshape(-1, 128, cols).abs().amax(1).repeat_interleave(128, 0)
    else:
        top = v.reshape(rows // 128, 128, cols // 128, 128).abs().amax((1, 3)).repeat_interleave(128, 0).repeat_interleave(128, 1)
    half, power = torch.frexp(top / 448.0)  # top / 448 = half * 2^power with half in [0.5, 1)
    e = torch.where(half == 0.5, power - 1, power).clamp(min=-127)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    q = torch.ldexp(v, -e.double())
    grain = torch.exp2((torch.frexp(q)[1] - 1).clamp(min=-6).double() - 3)  # three fraction bits; 2^-6 is the least normal
    return torch.ldexp((q / grain).round() * grain, e.double())[:x.shape[0], :x.shape[1]]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(dict(case, op="train") if case["op"] == "linear" else case, seed)
    finally:
        own = was
    if case["op"] in ("linear", "train"):
        # train's inputs are linear's and dy, which is made after the weight
        w = exact_q(s["w"], None)
        y = exact_q(s["x"], 1) @ w.t()
        if s["bias"] is not None:
            y = y + s["bias"].double()
        if case["op"] == "linear":
            return y
        dx = exact_q(s["dy"], 1) @ w
        dw = exact_q(s["dy"], 0).t() @ exact_q(s["x"], 0)
        return [y, dx, dw, None if s["bias"] is None else s["dy"].double().sum(0)]
    norm = torch.linalg.vector_norm(s["g"].double())
    clip = 1.0 / (norm + 1e-6) if float(norm) + 1e-6 > 1.0 else torch.ones_like(norm)
    if case["op"] == "norm":
        return [clip, norm]
    t = s["step"] + 1
    g = s["g"].double() * (clip if case["clip"] else s["scale"].double())
    m = 0.9 * s["m"].double() + 0.1 * g
    v = 0.999 * s["v"].double() + 0.001 * g ** 2
    step = (m / (1 - 0.9 ** t)) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
    p = s["p"].double()
    return [p - 1e-3 * 0.01 * p - 1e-3 * step, m, v]
