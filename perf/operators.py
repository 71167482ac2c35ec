"""The feed-forward half of a decoder layer around the quantised products, as measured cases.

Three operators: layer norm (forward, backward, and the step that keeps its normalised
input in 8 bits), activation checkpoints in 8 bits (saved and read back), and the gated
feed-forward product of quantised operands, h = act(x gate^T) * (x up^T) (alone, and as a
training step that keeps gate and up in 8 bits for its backward pass).  Hidden size 2048,
width 5632 and 16384 tokens are the block of this repository's benchmark.

With `own` false `run` computes each operator in elementary torch operations; with it true
it makes the calls a user makes of quantization_aware_amd.  `exact` is the operator's
definition in 64 bits.

The 8-bit checkpoint: blocks of 32 columns of a row share the power of two 2^(E - 133), E
the biased exponent of the block's largest magnitude; values are whole multiples of it up
to 127 (round to nearest even).
"""
import math

import torch

own = False

BLOCK = 32
EPS = 1e-5
# Clip scale over RMS of the b-bit midrise grid, a property of the inputs here.
ALPHA = {1: 0.7979, 2: 1.4935, 3: 2.0510, 4: 2.5134}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One token through a decoder layer's norm: the latency of a call.
        {"name": "norm_fwd_one_token", "op": "norm_fwd", "rows": 1, "cols": 2048, "x": "bf16", "w": "bf16"},
        # A training batch's forward norm, fp32 master parameters.
        {"name": "norm_fwd_16384x2048", "op": "norm_fwd", "rows": 16384, "cols": 2048, "x": "bf16", "w": "f32"},
        # Ragged sizes in fp32: rows that no vector width divides.
        {"name": "norm_bwd_1000x1111_f32", "op": "norm_bwd", "rows": 1000, "cols": 1111, "x": "f32", "w": "f32"},
        # The largest gradient of the benchmark's backward workload.
        {"name": "norm_bwd_65536x2048", "op": "norm_bwd", "rows": 65536, "cols": 2048, "x": "bf16", "w": "f32"},
        # A training step's norm with its normalised input kept in 8 bits.
        {"name": "norm_step8_16384x2048", "op": "norm_step8", "rows": 16384, "cols": 2048, "x": "bf16", "w": "bf16"},
        # The MLP intermediate of a training batch, checkpointed and read back.
        {"name": "act8_16384x5632", "op": "act8", "rows": 16384, "cols": 5632, "x": "bf16"},
        # A ragged fp32 activation whose last block is short.
        {"name": "act8_777x1001_f32", "op": "act8", "rows": 777, "cols": 1001, "x": "f32"},
        # One token of a frozen 4-bit model: the weights are the work.
        {"name": "gated_one_token", "op": "gated", "n": 1, "k": 2048, "m": 5632, "xb": 4, "wb": 4, "act": "silu", "out": "bf16"},
        # A decode batch.
        {"name": "gated_48_tokens", "op": "gated", "n": 48, "k": 2048, "m": 5632, "xb": 4, "wb": 4, "act": "silu", "out": "bf16"},
        # Ragged rows and width, mixed bit widths, fp32 output.
        {"name": "gated_300x1001_f32", "op": "gated", "n": 300, "k": 640, "m": 1001, "xb": 3, "wb": 2, "act": "gelu", "out": "f32"},
        # A long prompt batch through the frozen block.
        {"name": "gated_16384", "op": "gated", "n": 16384, "k": 2048, "m": 5632, "xb": 4, "wb": 4, "act": "silu", "out": "bf16"},
        # A training step of the block: forward with 8-bit checkpoints, then the gradients of gate and up.
        {"name": "gated_step_16384", "op": "gated_step", "n": 16384, "k": 2048, "m": 5632, "xb": 4, "wb": 4, "act": "silu", "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_step8", "act8", "gated", "gated", "gated_step"])
    if op.startswith("gated"):
        n = _log_int(rng, 1, 16384)
        k = 128 * _log_int(rng, 1, 64)
        m = _log_int(rng, 1, max(1, min(8192, 16384 * 2048 * 5632 // (n * k))))
        if rng.random() < 0.4:
            m = max(8, m // 8 * 8)
        while n * k * m > 16384 * 2048 * 5632 or n * m > 16384 * 5632:
            n = max(1, n // 2)
        return {"op": op, "n": n, "k": k, "m": m, "xb": rng.randint(1, 4), "wb": rng.randint(1, 4),
                "act": rng.choice(["silu", "gelu"]), "out": "bf16" if op == "gated_step" else rng.choice(["bf16", "f32"])}
    # (a norm of very few columns leaves its gradient to cancellation: x - mean spans what dy has)
    cols = _log_int(rng, 1 if op == "act8" else 16, 32768)
    if rng.random() < 0.4:
        cols = max(8, cols // 8 * 8)
    rows = _log_int(rng, 1, max(1, min(131072, (1 << 26) // cols)))
    case = {"op": op, "rows": rows, "cols": cols, "x": rng.choice(["bf16", "f32"])}
    if op != "act8":
        case["w"] = rng.choice(["bf16", "f32"])
    return case


def work(case):
    op = case["op"]
    if op.startswith("gated"):
        n, k, m = case["n"], case["k"], case["m"]
        o = 2 if case["out"] == "bf16" else 4
        read = n * k * case["xb"] / 8 + 2 * m * k * case["wb"] / 8 + 4 * (n + 2 * m)
        flops = 2.0 * n * k * 2 * m + 8.0 * n * m
        nbytes = read + n * m * o
        if op == "gated_step":  # gate and up in 8 bits written and read, dh read, both gradients written
            nbytes += 2 * 2 * n * m * (1 + 1 / BLOCK) + 3 * n * m * o
            flops += 16.0 * n * m
        return {"bytes": nbytes, "flops": flops}
    rows, cols = case["rows"], case["cols"]
    e = rows * cols
    x = 2 if case["x"] == "bf16" else 4
    kept = 1 + 1 / BLOCK
    if op == "act8":
        return {"bytes": e * (2 * x + 2 * kept), "flops": 4.0 * e}
    w = 2 if case["w"] == "bf16" else 4
    if op == "norm_fwd":
        return {"bytes": e * 2 * x + 8 * rows + 2 * cols * w, "flops": 8.0 * e}
    if op == "norm_bwd":
        return {"bytes": e * 3 * x + 8 * rows + 3 * cols * w, "flops": 14.0 * e}
    # the step: x read, y and the 8-bit copy written; dy and the copy read, dx written
    return {"bytes": e * (4 * x + 2 * kept) + 8 * rows + 5 * cols * w, "flops": 26.0 * e}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _activation(gen, rows, cols, device):
    """A residual stream: unit normal entries, a small offset, 1 column in 100 twenty times as large."""
    x = torch.randn((rows, cols), generator=gen, device=device) + 0.1
    x[:, ::100] *= 20.0
    return x


def _quantised(gen, rows, k, bits, std, device):
    """Codes (one a byte) and clip scales of normal rows of about `std`, as the quantiser's forward pass gives them."""
    y = torch.randn((rows, k), generator=gen, device=device)
    rms = std * torch.exp(0.25 * torch.randn((rows,), generator=gen, device=device))
    scale = ALPHA[bits] * rms
    u = torch.floor(y * ((2 ** bits - 1) / (2 * ALPHA[bits]))) + 2 ** (bits - 1)
    return u.clamp_(0, 2 ** bits - 1).to(torch.uint8), scale


def _pack(codes, bits):
    """One code a byte to the LSB-first stream of `bits` bits a code."""
    rows, k = codes.shape
    if bits == 8:
        return codes
    b = (codes.unsqueeze(-1) >> torch.arange(bits, dtype=torch.uint8, device=codes.device)) & 1
    b = b.reshape(rows, k * bits // 8, 8) << torch.arange(8, dtype=torch.uint8, device=codes.device)
    return b.sum(-1, dtype=torch.uint8).contiguous()


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    op = case["op"]
    if op.startswith("gated"):
        n, k, m, xb, wb = case["n"], case["k"], case["m"], case["xb"], case["wb"]
        st = dict(case)
        st["x"], st["x_scale"] = _quantised(gen, n, k, xb, 1.0, device)
        st["gate"], st["gate_scale"] = _quantised(gen, m, k, wb, k ** -0.5, device)
        st["up"], st["up_scale"] = _quantised(gen, m, k, wb, k ** -0.5, device)
        if op == "gated_step":
            st["dh"] = (1e-3 * torch.randn((n, m), generator=gen, device=device)).to(DTYPES[case["out"]])
        if own:
            # the operands that the quantiser writes for the same codes
            import quantization_aware_amd as qa

            st["x"] = qa.codes_to_operand(_pack(st["x"], xb), n, k, xb)
            st["gate"] = qa.codes_to_operand(_pack(st["gate"], wb), m, k, wb)
            st["up"] = qa.codes_to_operand(_pack(st["up"], wb), m, k, wb)
        return st
    rows, cols = case["rows"], case["cols"]
    xt = DTYPES[case["x"]]
    st = {"op": op, "x": _activation(gen, rows, cols, device).to(xt)}
    if op == "act8":
        return st
    wt = DTYPES[case["w"]]
    st["weight"] = (1 + 0.1 * torch.randn((cols,), generator=gen, device=device)).to(wt)
    st["bias"] = (0.1 * torch.randn((cols,), generator=gen, device=device)).to(wt)
    if op != "norm_fwd":
        st["dy"] = (1e-3 * torch.randn((rows, cols), generator=gen, device=device)).to(xt)
    if op == "norm_bwd":
        _, st["mean"], st["rstd"], _ = _norm_fwd(st["x"], st["weight"], st["bias"])
    return st


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _norm_fwd(x, weight, bias):
    xf = x.float()
    mean = xf.mean(1)
    c = xf - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + EPS)
    xhat = c * rstd[:, None]
    y = xhat * weight.float() + bias.float()
    return y.to(x.dtype), mean, rstd, xhat


def _norm_bwd(dy, xhat, rstd, weight):
    g = dy.float()
    a = g * weight.float()
    m1 = a.mean(1, keepdim=True)
    m2 = (a * xhat).mean(1, keepdim=True)
    dx = (a - m1 - xhat * m2) * rstd[:, None]
    return dx.to(dy.dtype), (g * xhat).sum(0).to(weight.dtype), g.sum(0).to(weight.dtype)


def _power_of_two(e):
    """2^e as doubles, for whole e of any normal double."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _act8(x):
    """The values of x's 8-bit checkpoint, fp32."""
    rows, cols = x.shape
    pad = -cols % BLOCK
    v = torch.nn.functional.pad(x.float(), (0, pad)).reshape(rows, -1, BLOCK)
    e = v.abs().amax(2, keepdim=True).view(torch.int32) >> 23
    q = torch.round(v.double() * _power_of_two(133 - e)).clamp(-127, 127)
    out = torch.where(e == 255, math.nan, q * _power_of_two(e - 133)).float()
    return out.reshape(rows, cols + pad)[:, :cols]


def _product(x, x_scale, xb, w, w_scale, wb):
    hx = x.float() - (2 ** xb - 1) / 2
    hw = w.float() - (2 ** wb - 1) / 2
    return (hx @ hw.t()) * ((x_scale * (2 / (2 ** xb - 1)))[:, None] * (w_scale * (2 / (2 ** wb - 1))))


def _act(g, act):
    return g / (1 + torch.exp(-g)) if act == "silu" else 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _act_slope(g, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * math.sqrt(0.5 / math.pi)


def _gated_bwd(dh, g, u, act):
    d = dh.float()
    return torch.cat([d * u * _act_slope(g, act), d * _act(g, act)], 1).to(dh.dtype)


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "norm_fwd":
        return _norm_fwd(st["x"], st["weight"], st["bias"])[:3]
    if op == "norm_bwd":
        xhat = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
        return _norm_bwd(st["dy"], xhat, st["rstd"], st["weight"])
    if op == "norm_step8":
        y, _, rstd, xhat = _norm_fwd(st["x"], st["weight"], st["bias"])
        return (y, *_norm_bwd(st["dy"], _act8(xhat), rstd, st["weight"]))
    if op == "act8":
        return _act8(st["x"]).to(st["x"].dtype)
    g = _product(st["x"], st["x_scale"], st["xb"], st["gate"], st["gate_scale"], st["wb"])
    u = _product(st["x"], st["x_scale"], st["xb"], st["up"], st["up_scale"], st["wb"])
    h = (_act(g, st["act"]) * u).to(DTYPES[st["out"]])
    if op == "gated":
        return h
    return h, _gated_bwd(st["dh"], _act8(g), _act8(u), st["act"])


def _run_own(st):
    import quantization_aware_amd as qa

    op = st["op"]
    if op == "norm_fwd":
        return qa.layer_norm_fwd(st["x"], st["weight"], st["bias"], EPS)[:3]
    if op == "norm_bwd":
        return qa.layer_norm_bwd(st["dy"], st["rstd"], st["weight"], x=st["x"], mean=st["mean"], bias_grad=True)
    if op == "norm_step8":
        y, _, rstd, kept = qa.layer_norm_fwd(st["x"], st["weight"], st["bias"], EPS, act8=True)
        return (y, *qa.layer_norm_bwd(st["dy"], rstd, st["weight"], act8=kept, bias_grad=True))
    if op == "act8":
        codes, scale = qa.act8_save(st["x"])
        return qa.act8_load(codes, scale, out_dtype=st["x"].dtype)
    train = op == "gated_step"
    h, gate8, up8 = qa.gated_fwd(st["x"], st["x_scale"], st["n"], st["xb"], st["gate"], st["gate_scale"], st["up"],
                                 st["up_scale"], st["m"], st["wb"], st["k"], act=st["act"],
                                 out_dtype=DTYPES[st["out"]], act8=train)
    if not train:
        return h
    return h, qa.gated_bwd(st["dh"], gate8, up8, act=st["act"])


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact8(x):
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        blk = x[:, c:c + BLOCK]
        _, e = torch.frexp(blk.abs().max(1, keepdim=True).values)  # the largest magnitude lies in [2^(e-1), 2^e)
        biased = torch.where(blk.abs().max(1, keepdim=True).values == 0, 0, (e + 126).clamp(min=0))
        step = torch.exp2((biased - 133).double())
        out[:, c:c + BLOCK] = torch.clamp(torch.round(blk / step), -127, 127) * step
    return out


def _exact_norm_bwd(dy, xhat, rstd, weight):
    c = dy.shape[1]
    dxhat = dy * weight
    dx = rstd[:, None] * (dxhat - dxhat.sum(1, keepdim=True) / c - xhat * ((dxhat * xhat).sum(1, keepdim=True) / c))
    return dx, torch.einsum("rc,rc->c", dy, xhat), dy.sum(0)


def _exact_phi(g):
    return 0.5 * torch.erfc(-g / math.sqrt(2.0))


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op.startswith("gated"):
        kx, kw = 2.0 / (2 ** case["xb"] - 1), 2.0 / (2 ** case["wb"] - 1)
        qx = (st["x"].double() - 0.5 * (2 ** case["xb"] - 1)) * (kx * st["x_scale"].double())[:, None]
        prod = []
        for w in ("gate", "up"):
            qw = (st[w].double() - 0.5 * (2 ** case["wb"] - 1)) * (kw * st[w + "_scale"].double())[:, None]
            prod.append(torch.matmul(qx, qw.t()))
            del qw
        g, u = prod
        silu = case["act"] == "silu"
        h = (g * torch.sigmoid(g) if silu else g * _exact_phi(g)) * u
        if op == "gated":
            return h
        g, u, d = _exact8(g), _exact8(u), st["dh"].double()
        if silu:
            s = torch.sigmoid(g)
            value, slope = g * s, s + g * s * torch.sigmoid(-g)
        else:
            value = g * _exact_phi(g)
            slope = _exact_phi(g) + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
        return h, torch.cat([d * u * slope, d * value], 1)
    x = st["x"].double()
    if op == "act8":
        return _exact8(x)
    weight, bias = st["weight"].double(), st["bias"].double()
    if op == "norm_bwd":
        rstd = st["rstd"].double()
        return _exact_norm_bwd(st["dy"].double(), (x - st["mean"].double()[:, None]) * rstd[:, None], rstd, weight)
    mean = x.sum(1) / x.shape[1]
    rstd = ((x - mean[:, None]).square().sum(1) / x.shape[1] + EPS).rsqrt()
    xhat = (x - mean[:, None]) * rstd[:, None]
    y = torch.addcmul(bias, xhat, weight)
    if op == "norm_fwd":
        return y, mean, rstd
    return (y, *_exact_norm_bwd(st["dy"].double(), _exact8(xhat), rstd, weight))
