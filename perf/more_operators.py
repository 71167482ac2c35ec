"""Products in 8-bit integers and the mixture-of-experts layer built on them, as measured cases.

Three operators: the product of two tensors held in 8-bit integers with a scale for each token and each
channel (gemm8), a linear layer that quantises its input to such integers and multiplies it by a kept
weight (linear8) or, in training, quantises both and gives the gradients (step), and a whole mixture-of-experts layer for a few tokens: routing, the chosen experts' gated
products, the quantisation between them and the way back, summed over the experts (moe).  Widths of 2048
and 5632 and batches of 16384 tokens are the block of this repository's benchmark.

With `own` false `run` computes each operator in elementary torch operations; with it true it makes the
calls a user makes of quantization_aware_amd.  `exact` is the operator's definition in 64 bits.

What an integer stands for: a row of b-bit codes c in [-2^(b-1), 2^(b-1) - 1] with clip scale s has the
values (2 c + 1) s / (2^b - 1).  The quantiser of a row: an orthonormal Hadamard transform of each block
of columns, s = ALPHA[b] times the row's root mean square, and c = floor(y / step) with step =
2 s / (2^b - 1), clipped.  The gradient passes where y is no further than half a step beyond the outermost
value, and comes back through the same transform.  Codes of up to 8 bits lie one in a byte; the experts' 4-bit weights lie two in
a byte, the even column in the low half, as c + 8.
"""
import math

import torch

own = False

# The clip scale over the root mean square that has the least squared error on a normal variable.
ALPHA = {1: 0.7978845608028653, 2: 1.4935300289152593, 3: 2.0510680450522036, 4: 2.514004591499794,
         5: 2.9161512493387267, 6: 3.2779847974234526, 7: 3.6110971962796867, 8: 3.9222044167461094}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST = 16384 * 2048 * 5632  # products of the largest listed matrix product
MOST_EXPERTS = 128 * 768 * 2048  # entries of the largest listed set of one projection's weights


def listed():
    return [
        # One token through an attention projection: the latency of a call.
        {"name": "gemm8_one_token", "op": "gemm8", "n": 1, "k": 2048, "m": 2048, "xb": 8, "wb": 8, "out": "bf16"},
        # A decode batch through the up projection: the weights are the work.
        {"name": "gemm8_48_tokens", "op": "gemm8", "n": 48, "k": 2048, "m": 5632, "xb": 8, "wb": 8, "out": "bf16"},
        # Ragged rows, columns and inner size, mixed widths, fp32 output.
        {"name": "gemm8_333x1001_f32", "op": "gemm8", "n": 333, "k": 960, "m": 1001, "xb": 7, "wb": 5, "out": "f32"},
        # A prompt through the down projection.
        {"name": "gemm8_2048_down", "op": "gemm8", "n": 2048, "k": 5632, "m": 2048, "xb": 8, "wb": 8, "out": "bf16"},
        # A training batch through the up projection.
        {"name": "gemm8_16384_up", "op": "gemm8", "n": 16384, "k": 2048, "m": 5632, "xb": 8, "wb": 8, "out": "bf16"},
        # A few tokens of a frozen 8-bit layer, fp32 activations: quantise, multiply.
        {"name": "linear8_5_tokens_f32", "op": "linear8", "n": 5, "k": 5632, "m": 2048, "block": 256, "x": "f32", "xb": 8, "wb": 8, "step": False},
        # A training step of the output projection: forward, and the gradients of input and weight.
        {"name": "linear8_step_16384", "op": "linear8", "n": 16384, "k": 2048, "m": 2048, "block": 128, "x": "bf16", "xb": 8, "wb": 8, "step": True},
        # One token through an expert layer of 4-bit weights: latency, and the chosen experts' weights.
        {"name": "moe_one_token", "op": "moe", "n": 1, "e": 64, "top": 8, "k": 2048, "m": 1024, "xb": 4, "wb": 4, "hb": 4, "block": 128, "act": "silu", "logits": "f32", "all": False},
        # Odd counts of tokens and experts, widths that end inside a tile, 5-bit weights, weights of all experts' softmax.
        {"name": "moe_7_ragged", "op": "moe", "n": 7, "e": 13, "top": 3, "k": 704, "m": 448, "xb": 6, "wb": 5, "hb": 6, "block": 64, "act": "gelu", "logits": "bf16", "all": True},
        # A small decode batch: half of the experts are chosen by some token.
        {"name": "moe_16_tokens", "op": "moe", "n": 16, "e": 64, "top": 8, "k": 2048, "m": 1024, "xb": 8, "wb": 4, "hb": 8, "block": 128, "act": "silu", "logits": "f32", "all": False},
        # A decode batch over a few wide experts in 8 bits: many tokens an expert.
        {"name": "moe_64_wide_8bit", "op": "moe", "n": 64, "e": 8, "top": 2, "k": 2048, "m": 5632, "xb": 8, "wb": 8, "hb": 8, "block": 128, "act": "silu", "logits": "bf16", "all": False},
        # A decode batch over many narrow experts: all their weights, a few tokens each.
        {"name": "moe_64_of_128", "op": "moe", "n": 64, "e": 128, "top": 8, "k": 2048, "m": 768, "xb": 8, "wb": 4, "hb": 8, "block": 256, "act": "silu", "logits": "f32", "all": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemm8", "gemm8", "linear8", "moe", "moe"])
    if op == "moe":
        block = rng.choice([64, 128, 256])
        e = _log_int(rng, 2, 128)
        k = 64 * _log_int(rng, 2, 64)
        m = block * _log_int(rng, 1, 5632 // block)
        while e * k * m > MOST_EXPERTS:
            m, k = max(block, m // 2 // block * block), max(64, k // 2 // 64 * 64)
        wb = rng.choice([4, 4, 8, rng.randint(1, 8)])
        return {"op": op, "n": _log_int(rng, 1, 64), "e": e, "top": rng.randint(1, min(8, e)), "k": k, "m": m,
                "xb": rng.choice([4, 8, rng.randint(2, 8)]), "wb": wb, "hb": rng.choice([4, 8, rng.randint(3, 8)]),
                "block": block, "act": rng.choice(["silu", "gelu"]), "logits": rng.choice(["f32", "bf16"]),
                "all": rng.random() < 0.3}
    block = rng.choice([64, 128, 256])
    n = _log_int(rng, 1, 16384)
    k = block * _log_int(rng, 1, 8192 // block) if op == "linear8" else 64 * _log_int(rng, 1, 128)
    m = _log_int(rng, 1, 8192)
    if rng.random() < 0.4:
        m = max(8, m // 8 * 8)
    while n * k * m > MOST or n * m > 16384 * 5632:
        n = max(1, n // 2)
    xb, wb = rng.choice([8, rng.randint(1, 8)]), rng.choice([8, rng.randint(1, 8)])
    if op == "linear8":
        step = rng.random() < 0.4
        if step:  # three products
            n = max(1, min(n, MOST // 3 // (k * m)))
        return {"op": op, "n": n, "k": k, "m": m, "block": block, "x": "bf16" if step else rng.choice(["bf16", "f32"]),
                "xb": max(xb, 4), "wb": max(wb, 2), "step": step}
    return {"op": op, "n": n, "k": k, "m": m, "xb": xb, "wb": wb, "out": rng.choice(["bf16", "f32"])}


def work(case):
    n, k, m = case["n"], case["k"], case["m"]
    if case["op"] == "moe":
        e, top = case["e"], case["top"]
        chosen = e * (1 - (1 - top / e) ** n)  # experts that some token takes, on average
        weights = chosen * (3 * m * k * (0.5 if case["wb"] == 4 else 1.0) + 4 * (2 * m + k))
        logits = n * e * (2 if case["logits"] == "bf16" else 4)
        return {"bytes": weights + n * (k + 4) + logits + n * k * 2, "flops": 6.0 * n * top * m * k}
    x = 1 if case["op"] == "gemm8" else 2 if case["x"] == "bf16" else 4
    out = 4 if case.get("out") == "f32" else 2
    if case.get("step"):  # x, w and dy read, y, dx and dw written
        return {"bytes": 4.0 * (n * k + m * k + n * m), "flops": 6.0 * n * k * m}
    return {"bytes": n * k * x + m * k + 4.0 * (n + m) + n * m * out, "flops": 2.0 * n * k * m}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _quantised(gen, shape, bits, std, device):
    """Codes and clip scales of normal rows of about `std`, as the quantiser gives them."""
    y = torch.randn(shape, generator=gen, device=device)
    rms = std * torch.exp(0.25 * torch.randn(shape[:-1], generator=gen, device=device))
    half = 2 ** (bits - 1)
    c = torch.floor(y.mul_((2 ** bits - 1) / (2 * ALPHA[bits]))).clamp_(-half, half - 1).to(torch.int8)
    return c, ALPHA[bits] * rms


def _experts(gen, shape, bits, device):
    c, scale = _quantised(gen, shape, bits, shape[-1] ** -0.5, device)
    if bits == 4:
        u = (c + 8).to(torch.uint8)
        c = u[..., 0::2] | (u[..., 1::2] << 4)
    return c, scale


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    n, k, m = case["n"], case["k"], case["m"]
    st = dict(case)
    if case["op"] == "moe":
        e = case["e"]
        st["x"], st["x_scale"] = _quantised(gen, (n, k), case["xb"], 1.0, device)
        st["router"] = torch.randn((n, e), generator=gen, device=device).to(DTYPES[case["logits"]])
        st["gate"], st["gate_scale"] = _experts(gen, (e, m, k), case["wb"], device)
        st["up"], st["up_scale"] = _experts(gen, (e, m, k), case["wb"], device)
        st["down"], st["down_scale"] = _experts(gen, (e, k, m), case["wb"], device)
        return st
    if case.get("step"):
        st["w"] = (k ** -0.5 * torch.randn((m, k), generator=gen, device=device)).to(torch.bfloat16)
        st["dy"] = (1e-3 * torch.randn((n, m), generator=gen, device=device)).to(torch.bfloat16)
    else:
        st["w"], st["w_scale"] = _quantised(gen, (m, k), case["wb"], k ** -0.5, device)
    if case["op"] == "gemm8":
        st["x"], st["x_scale"] = _quantised(gen, (n, k), case["xb"], 1.0, device)
    else:  # a residual stream: 1 column in 100 twenty times as large
        x = torch.randn((n, k), generator=gen, device=device)
        x[:, ::100] *= 20.0
        st["x"] = x.to(DTYPES[case["x"]])
    return st


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _odd(c, bits):
    """2 c + 1 of a tensor's codes, in fp32."""
    if c.dtype == torch.uint8:
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2).to(torch.int8) - 8
    return c.float() * 2 + 1


def _step(scale, bits):
    return scale * (1 / (2 ** bits - 1))


def _hadamard(block, device, dtype=torch.float32):
    i = torch.arange(block, device=device)
    bits = (i[:, None] & i[None, :])
    parity = sum((bits >> s) & 1 for s in range(8)) & 1
    return (1 - 2 * parity).to(dtype) * block ** -0.5


def _quantise(x, block, bits):
    """2 c + 1, half the step of the rows of x on the bits' grid, and where the gradient passes."""
    xf = x.float()
    y = (xf.unflatten(-1, (-1, block)) @ _hadamard(block, x.device)).flatten(-2)
    step = ALPHA[bits] * torch.sqrt((xf * xf).mean(-1)) * (1 / (2 ** bits - 1))
    half = 2 ** (bits - 1)
    c = torch.floor(y / (2 * step[..., None])).nan_to_num(0.0).clamp(-half, half - 1)
    return 2 * c + 1, step, y.abs() <= step[..., None] * 2 ** bits


def _act(g, act):
    return g / (1 + torch.exp(-g)) if act == "silu" else 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _route(logits, top, over_all):
    """The experts of each token, the largest logits first (of equal ones the lowest index), and their weights."""
    l = logits.float()
    value, index = torch.sort(l, dim=-1, descending=True, stable=True)
    p = torch.exp(value - value[:, :1])
    p = p[:, :top] / (p if over_all else p[:, :top]).sum(-1, keepdim=True)
    return index[:, :top], p


def _moe(st):
    n, e, top, k = st["n"], st["e"], st["top"], st["k"]
    index, p = _route(st["router"], top, st["all"])
    if n * top < e:  # a batch entry for each token and chosen expert
        pick, rows = index.reshape(-1), torch.arange(n, device=index.device).repeat_interleave(top)[:, None]
    else:  # one for each expert, with all tokens
        pick, rows = torch.arange(e, device=index.device), torch.arange(n, device=index.device).expand(e, n)
    x, xs = _odd(st["x"], st["xb"])[rows], _step(st["x_scale"], st["xb"])[rows]

    def product(a, a_step, name):
        w = _odd(st[name][pick], st["wb"])
        return torch.matmul(a, w.transpose(1, 2).contiguous()) * (a_step[..., None] * _step(st[name + "_scale"][pick], st["wb"])[:, None])

    h = _act(product(x, xs, "gate"), st["act"]) * product(x, xs, "up")
    y = product(*_quantise(h, st["block"], st["hb"])[:2], "down")
    if n * top < e:
        return (y.reshape(n, top, k) * p[..., None]).sum(1).to(torch.bfloat16)
    share = torch.zeros((n, e), device=p.device).scatter_(1, index, p)
    return (y * share.t()[..., None]).sum(0).to(torch.bfloat16)


def _step_of(st):
    """The layer's output and the gradients of x and w."""
    (x, xs, x_passes), (w, ws, w_passes) = _quantise(st["x"], st["block"], st["xb"]), _quantise(st["w"], st["block"], st["wb"])
    y = (x @ w.t()) * (xs[:, None] * ws)
    dy = st["dy"].float()
    turn = _hadamard(st["block"], dy.device)

    def back(g, passes):
        return ((g * passes).unflatten(-1, (-1, st["block"])) @ turn).flatten(-2).to(torch.bfloat16)

    return y.to(torch.bfloat16), back((dy * ws) @ w, x_passes), back((dy * xs[:, None]).t() @ x, w_passes)


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "moe":
        return _moe(st)
    if st.get("step"):
        return _step_of(st)
    if st["op"] == "gemm8":
        x, x_step = _odd(st["x"], st["xb"]), _step(st["x_scale"], st["xb"])
    else:
        x, x_step, _ = _quantise(st["x"], st["block"], st["xb"])
    y = (x @ _odd(st["w"], st["wb"]).t()) * (x_step[:, None] * _step(st["w_scale"], st["wb"]))
    return y.to(DTYPES[st.get("out", "bf16")])


def _run_own(st):
    import quantization_aware_amd as qa

    if st["op"] == "moe":
        return qa.moe_fwd(st["x"], st["x_scale"], st["xb"], st["router"], st["gate"], st["gate_scale"], st["up"],
                          st["up_scale"], st["down"], st["down_scale"], st["wb"], st["top"], block=st["block"],
                          h_bits=st["hb"], act=st["act"], over_all=st["all"], out_dtype=torch.bfloat16)
    if st.get("step"):
        from quantization_aware_amd.linear import quest_linear

        x, w = st["x"].detach().requires_grad_(), st["w"].detach().requires_grad_()
        y = quest_linear(x, w, block=st["block"], bits_x=st["xb"], bits_w=st["wb"], int8=True)
        return (y.detach(), *torch.autograd.grad(y, (x, w), st["dy"]))
    x, x_scale = st["x"], st.get("x_scale")
    if st["op"] == "linear8":
        x, x_scale, _ = qa.quantize_fwd_i8(x, st["block"], st["xb"])
    return qa.gemm_i8(x, x_scale, st["xb"], st["w"], st["w_scale"], st["wb"], out_dtype=DTYPES[st.get("out", "bf16")])


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_values(c, scale, bits):
    """The values that codes stand for."""
    if c.dtype == torch.uint8:
        wide = torch.empty(c.shape[:-1] + (2 * c.shape[-1],), dtype=torch.float64, device=c.device)
        wide[..., 0::2] = torch.remainder(c, 16)
        wide[..., 1::2] = torch.div(c, 16, rounding_mode="floor")
        wide -= 8
    else:
        wide = c.double()
    return (wide + 0.5) * (scale.double() * (2.0 / (2 ** bits - 1)))[..., None]


def _exact_transform(x, block):
    y = x.reshape(-1, block)
    half = 1
    while half < block:  # the transform's butterflies
        y = y.reshape(-1, block // (2 * half), 2, half)
        y = torch.stack((y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]), 2)
        half *= 2
    return y.reshape(x.shape) / math.sqrt(block)


def _exact_quantised(x, block, bits):
    """The values of the rows of x on the bits' grid, and where the gradient passes."""
    x = x.double()
    y = _exact_transform(x, block)
    scale = ALPHA[bits] * x.square().mean(1).sqrt()
    step = (2.0 * scale / (2 ** bits - 1))[:, None]
    level = torch.clamp(torch.floor(y / step), -2 ** (bits - 1), 2 ** (bits - 1) - 1)
    passes = y.abs() <= scale[:, None] + step / 2
    return torch.where(step > 0, (level + 0.5) * step, 0.0), passes


def exact(case, seed):
    st = prepare(case, seed)
    if case.get("step"):
        dy, block = st["dy"].double(), case["block"]
        (x, x_passes), (w, w_passes) = _exact_quantised(st["x"], block, case["xb"]), _exact_quantised(st["w"], block, case["wb"])
        return (torch.matmul(x, w.t()), _exact_transform(torch.where(x_passes, torch.matmul(dy, w), 0.0), block),
                _exact_transform(torch.where(w_passes, torch.matmul(dy.t(), x), 0.0), block))
    if case["op"] != "moe":
        x = _exact_values(st["x"], st["x_scale"], case["xb"]) if case["op"] == "gemm8" else _exact_quantised(st["x"], case["block"], case["xb"])[0]
        return torch.matmul(x, _exact_values(st["w"], st["w_scale"], case["wb"]).t())
    x = _exact_values(st["x"], st["x_scale"], case["xb"])
    logits = st["router"].double()
    out = torch.zeros((case["n"], case["k"]), dtype=torch.float64, device=x.device)
    # an expert is chosen where fewer than `top` others come before it
    ahead = (logits[:, :, None] < logits[:, None, :]).sum(2)
    same = logits[:, :, None] == logits[:, None, :]
    ahead += torch.tril(same, -1).sum(2)
    chosen = ahead < case["top"]
    share = torch.softmax(logits if case["all"] else logits.masked_fill(~chosen, -math.inf), 1)
    for e in range(case["e"]):
        t = torch.nonzero(chosen[:, e]).flatten()
        if not t.numel():
            continue
        g, u = (x[t] @ _exact_values(st[w][e], st[w + "_scale"][e], case["wb"]).t() for w in ("gate", "up"))
        h = (g * torch.sigmoid(g) if case["act"] == "silu" else g * 0.5 * torch.erfc(-g / math.sqrt(2.0))) * u
        q, _ = _exact_quantised(h, case["block"], case["hb"])
        out[t] += share[t, e][:, None] * (q @ _exact_values(st["down"][e], st["down_scale"][e], case["wb"]).t())
    return out
