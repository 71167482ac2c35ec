"""Gradients of the quantised layers: whose memory they hold, and those of QuestMoE against 64 bits."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import moe_oracle as mo
import quantization_aware_amd as qa
from oracle import quest_oracle as qo
from quantization_aware_amd.experts import QuestMoE, route
from quantization_aware_amd.linear import QuestLinear, quest_linear, quest_linear_int8

pytestmark = pytest.mark.gpu

U = mo.U  # half a step of fp32, relative


def log(msg: str) -> None:
    print(f"[gpu-int8-gradients] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    return torch.device("cuda", 0)


TYPES = [(torch.bfloat16, torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32, torch.bfloat16),
         (torch.float32, torch.bfloat16, torch.float32), (torch.float32, torch.float32, torch.float32)]


def owns(grad):
    return grad.untyped_storage().nbytes() == grad.numel() * grad.element_size()


@pytest.mark.parametrize("x_dtype,w_dtype,compute", TYPES)
@pytest.mark.parametrize("n,bits_x,bits_w", [(64, 8, 8), (64, 4, 4), (63, 8, 8), (64, 8, 6)])
def test_gradients_hold_their_own_memory(dev, x_dtype, w_dtype, compute, n, bits_x, bits_w):
    """weight.grad outlives the step: it keeps nothing alive but itself, however x's and w's codes are laid out."""
    log(f"memory of gradients n={n} {bits_x} and {bits_w} bits {x_dtype} {w_dtype} {compute}")
    x = torch.randn(n, 256, device=dev).to(x_dtype).requires_grad_()
    w = torch.randn(24, 256, device=dev).to(w_dtype).requires_grad_()
    quest_linear(x, w, bits_x=bits_x, bits_w=bits_w, compute_dtype=compute, int8=True).float().sum().backward()
    for t in (x, w):
        assert t.grad.dtype == t.dtype and t.grad.shape == t.shape and owns(t.grad)


@pytest.mark.parametrize("x_dtype,w_dtype,compute", TYPES)
@pytest.mark.parametrize("n", [64, 63])
def test_gradients_of_the_default_layer_hold_their_own_memory(dev, x_dtype, w_dtype, compute, n):
    """The same of the FP6 product's layer, whose codes are the rows of one tensor where n is a multiple of 4."""
    x = torch.randn(n, 256, device=dev).to(x_dtype).requires_grad_()
    w = torch.randn(24, 256, device=dev).to(w_dtype).requires_grad_()
    quest_linear(x, w, bits_x=4, bits_w=4, compute_dtype=compute).float().sum().backward()
    for t in (x, w):
        assert t.grad.dtype == t.dtype and t.grad.shape == t.shape and owns(t.grad)


# ---------------------------------------------------------------------------
# The experts
# ---------------------------------------------------------------------------

class Bounded:
    """Values in 64 bits with what an fp32 evaluation of them may be off by, entry by entry."""

    def __init__(self, v, err=None):
        self.v = np.asarray(v, np.float64)
        self.err = np.zeros_like(self.v) if err is None else err

    def __matmul__(self, o):
        """A sum of products: each product one rounding, each addition one."""
        size = np.abs(self.v) @ np.abs(o.v)
        err = self.err @ (np.abs(o.v) + o.err) + np.abs(self.v) @ o.err
        return Bounded(self.v @ o.v, err + (self.v.shape[1] + 1) * U * (size + err))

    def __mul__(self, o):
        err = self.err * (np.abs(o.v) + o.err) + np.abs(self.v) * o.err
        v = self.v * o.v
        return Bounded(v, err + U * (np.abs(v) + err))

    def __add__(self, o):
        v = self.v + o.v
        err = self.err + o.err
        return Bounded(v, err + U * (np.abs(v) + err))

    def t(self):
        return Bounded(self.v.T, self.err.T)

    def rows(self, i):
        return Bounded(self.v[i], self.err[i])

    def back(self, mask, block):
        """The trust backward: masked, log2(block) additions and a scaling."""
        v, err = self.v * mask, self.err * mask

        def mix(a):
            return np.repeat(np.abs(a).reshape(len(a), -1, block).sum(-1) / math.sqrt(block), block, 1)

        return Bounded(qo.blockwise_hadamard(v, block), mix(err) + (math.log2(block) + 3) * U * (mix(v) + mix(err)))


def quantised(t, block, bits):
    """The values and the trust mask of the layer's own quantiser, values as the layer rebuilds them in fp32."""
    c, s, m = qa.quantize_fwd_i8(t.detach().contiguous(), block, bits, trust=1.3 if bits == 1 else 1.0, with_mask=True)
    v = mo.values(c.cpu().numpy().astype(np.float64), s.cpu().numpy(), bits)
    return Bounded(v, 3 * U * np.abs(v)), qo.unpack_lsb_first(m.cpu().numpy(), 1, t.shape[1]).astype(np.float64)


def activation(g, name):
    """act(g) and act'(g).  fp32 evaluations of both, with g's own error e: |act'| and |act''| stay below 1.2, and what
    the function is off by is counted as 16 roundings of |g| (the value) and of 1 + |g| (the slope)."""
    x = g.v
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-x))
        v, d = x * s, s * (1.0 + x * (1.0 - s))
    else:
        phi = 0.5 * mo.erfc(-x / math.sqrt(2.0))
        v, d = x * phi, phi + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    return Bounded(v, 1.2 * g.err + 16 * U * np.abs(x)), Bounded(d, 1.2 * g.err + 16 * U * (1.0 + np.abs(x)))


@pytest.mark.parametrize("act,over_all,bits", [("silu", False, (8, 8, 8)), ("gelu", True, (8, 8, 8)),
                                               ("silu", True, (6, 4, 5)), ("gelu", False, (4, 4, 4))])
def test_experts_gradients(dev, act, over_all, bits):
    """x's, the router's and both weights' gradients, entry by entry, from the layer's own codes and masks.

    Expert 4 is taken by no token: its gradients are zeros."""
    bx, bw, bh = bits
    n, k, m, e, top, block = 25, 128, 64, 6, 2, 64
    log(f"experts {act} over_all={over_all} bits {bits}")
    torch.manual_seed(3)
    moe = QuestMoE(k, m, e, top, block=block, bits_x=bx, bits_w=bw, bits_h=bh, compute_dtype=torch.float32, act=act,
                   over_all=over_all, device=dev)
    x = torch.randn(n, k, device=dev)
    x[:, 0] = 3.0
    with torch.no_grad():
        moe.router[4].zero_()
        moe.router[4, 0] = -20.0  # a logit of -60
    x.requires_grad_()
    dout = torch.randn(n, k, device=dev)
    y = moe(x)
    dx, dr, dgu, dd = torch.autograd.grad(y, (x, moe.router, moe.gate_up, moe.down), dout)
    with torch.no_grad():
        logits = torch.nn.functional.linear(x, moe.router)
        weight, index = route(logits, top, over_all)
        p = [t.cpu().numpy() for t in (weight.double(), index)]
    assert not (p[1] == 4).any()
    # (the logits and weights are the layer's own: the same calls on the same inputs)
    qx, mx = quantised(x, block, bx)
    d_out = Bounded(dout.double().cpu().numpy())
    want_x = Bounded(np.zeros((n, k)))
    d_weight = Bounded(np.zeros((n, top)))
    want_y = Bounded(np.zeros((n, k)))
    for i in range(e):
        token, rank = np.nonzero(p[1] == i)
        if not len(token):
            assert (dgu[i] == 0).all() and (dd[i] == 0).all()
            continue
        at = torch.from_numpy(token).to(dev)
        qw, mw = quantised(moe.gate_up[i], block, bw)
        qd, md = quantised(moe.down[i], block, bw)
        # h as the layer has it, bit by bit: its codes are the layer's
        with torch.no_grad():
            g32, u32 = quest_linear(x.detach()[at], moe.gate_up[i], block=block, bits_x=bx, bits_w=bw,
                                    compute_dtype=torch.float32, int8=True).chunk(2, -1)
            h32 = (torch.nn.functional.silu(g32) if act == "silu" else torch.nn.functional.gelu(g32)) * u32
        qh, mh = quantised(h32, block, bh)
        rows = Bounded(qx.v[token], qx.err[token])
        gu = qx.v[token] @ qw.v.T
        g, u = (Bounded(v, 8 * U * np.abs(v)) for v in (gu[:, :m], gu[:, m:]))
        a, slope = activation(g, act)
        down = qh.v @ qd.v.T
        down = Bounded(down, 8 * U * np.abs(down))
        share = Bounded(p[0][token, rank][:, None])
        dw = (down * d_out.rows(token)) @ Bounded(np.ones((k, 1)))
        d_weight.v[token, rank], d_weight.err[token, rank] = dw.v[:, 0], dw.err[:, 0]
        part = down * share
        want_y.v[token] += part.v
        want_y.err[token] += part.err + top * U * np.abs(part.v)
        dy = d_out.rows(token) * share
        check(f"down {i}", dd[i], (dy.t() @ qh).back(md, block))
        dh = (dy @ qd).back(mh, block)
        dg, du = dh * u * slope, dh * a
        both = Bounded(np.concatenate([dg.v, du.v], 1), np.concatenate([dg.err, du.err], 1))
        check(f"gate_up {i}", dgu[i], (both.t() @ rows).back(mw, block))
        part = (both @ qw).back(mx[token], block)
        want_x.v[token] += part.v
        want_x.err[token] += part.err + (top + 1) * U * np.abs(part.v)
    check("y", y.detach(), want_y)
    # the router: softmax over the chosen or over all logits, then its linear layer
    l64 = logits.double().cpu().numpy()
    d_logits = np.zeros((n, e))
    d_err = np.zeros((n, e))
    for t in range(n):
        over = np.arange(e) if over_all else p[1][t]
        soft = np.exp(l64[t, over] - l64[t, over].max())
        soft /= soft.sum()
        d = np.zeros(len(over))
        size = np.zeros(len(over))
        for r in range(top):
            j = int(np.nonzero(over == p[1][t, r])[0][0])
            d[j] += d_weight.v[t, r]
            size[j] += d_weight.err[t, r]
        d_logits[t, over] = soft * (d - (soft * d).sum())
        off = (e + 8) * U  # of soft, relative: two exponentials, their sum and a quotient
        d_err[t, over] = soft * (size + (soft * size).sum()) + soft * (np.abs(d) + (soft * np.abs(d)).sum()) * (3 * off + (e + 4) * U)
    d_logits = Bounded(d_logits, d_err)
    check("router", dr, d_logits.t() @ Bounded(x.detach().double().cpu().numpy()))
    check("x", dx, want_x + d_logits @ Bounded(moe.router.detach().double().cpu().numpy()))


def check(name, got, want):
    got = got.double().cpu().numpy()
    ratio = np.abs(got - want.v) / (want.err * (1 + U) + 1e-30)
    assert got.shape == want.v.shape and (ratio <= 1).all(), f"{name}: {ratio.max():.3g} of the bound"
    # (the bound is a check at all: a gradient off by a quarter of its size would not pass)
    assert np.linalg.norm(want.err) < 0.25 * np.linalg.norm(want.v), name
    log(f"{name}: {ratio.max():.3g} of the bound, {np.linalg.norm(want.err) / np.linalg.norm(want.v):.2g} of the size")


@pytest.mark.parametrize("over_all", [False, True])
def test_logits_of_minus_infinity(dev, over_all):
    """Trained and frozen alike: such an expert is not taken, and a token without any gives zeros and no gradient."""
    torch.manual_seed(4)
    moe = QuestMoE(128, 64, 4, 2, block=64, bits_x=8, bits_w=8, compute_dtype=torch.float32, over_all=over_all, device=dev)
    x = torch.randn(5, 128, device=dev)
    with torch.no_grad():
        moe.router[:, 0] = torch.tensor([-1e30, -1e30, -1e30, -1e30])
        moe.router[:, 1] = torch.tensor([0.0, 0.0, 0.0, -1e30])
        x[:, :2] = 0.0
        x[1, 0] = 1e10  # every logit -infinity
        x[3, 1] = 1e10  # that of expert 3
    x.requires_grad_()
    y = moe(x)
    assert (y[1] == 0).all() and y.isfinite().all()
    y.sum().backward()
    # (token 3 has y of about 1e18 and so have its logits' gradients: by the router's -1e30 they pass fp32's range)
    assert x.grad[[0, 1, 2, 4]].isfinite().all() and all(p.grad.isfinite().all() for p in moe.parameters())
    assert (x.grad[1] == 0).all()
    frozen = moe.freeze()(x.detach())
    assert (frozen[1] == 0).all()
    # (h keeps fp32 on both sides: only codes at a level's edge differ)
    assert float((frozen - y.detach()).norm() / frozen.norm()) < 0.02


# ---------------------------------------------------------------------------
# The frozen linear layer beside the trained one
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_frozen_outputs_carry_no_gradient(dev, bias, dtype):
    layer = QuestLinear(256, 96, bias=bias, bits_x=8, bits_w=8, compute_dtype=dtype, int8=True, device=dev).freeze()
    x = torch.randn(3, 256, device=dev, requires_grad=True)
    y = layer(x)
    assert not y.requires_grad and y.grad_fn is None
    codes, scale = layer._w_operand, layer._w_scale
    assert not quest_linear_int8(x, codes, scale, 8, bias=layer.bias, out_dtype=dtype).requires_grad


@pytest.mark.parametrize("compute", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bias", [True, False])
def test_frozen_outputs_have_the_trained_type(dev, compute, bias):
    layer = QuestLinear(256, 96, bias=bias, bits_x=8, bits_w=8, compute_dtype=compute, int8=True, device=dev)
    if bias:
        torch.nn.init.normal_(layer.bias)
    x = torch.randn(3, 5, 256, device=dev)
    with torch.no_grad():
        want = layer(x)
    got = layer.freeze()(x)
    assert want.dtype == got.dtype == compute and torch.equal(got, want)
