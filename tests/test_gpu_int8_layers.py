"""QuestLinear with products in 8-bit integers and QuestMoE: values and gradients against the definitions, their frozen
forms, the calls together as a decoder layer uses them, streams and HIP graphs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_oracle as mo
import quantization_aware_amd as qa
from oracle import quest_oracle as qo
from quantization_aware_amd.experts import QuestMoE, route
from quantization_aware_amd.feedforward import layer_norm
from quantization_aware_amd.linear import QuestLinear, quest_linear, quest_linear_int8

pytestmark = pytest.mark.gpu


def log(msg: str) -> None:
    print(f"[gpu-int8-layers] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    return torch.device("cuda", 0)


def rand(shape, seed, dtype, dev, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=g)).to(dtype).to(dev)


def hadamard(x: np.ndarray, block: int) -> np.ndarray:
    return qo.blockwise_hadamard(x, block)


# ---------------------------------------------------------------------------
# The linear layer
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,k,m,block,bx,bw", [(8, 256, 40, 128, 8, 8), (37, 192, 72, 64, 8, 8), (5, 512, 33, 256, 6, 8),
                                               (64, 384, 130, 128, 4, 4), (12, 128, 16, 128, 1, 1), (300, 320, 96, 64, 7, 5)])
def test_linear_gradients(dev, n, k, m, block, bx, bw):
    """y and the gradients in fp32 from the layer's own codes and masks, in 64 bits."""
    log(f"linear {n}x{k}x{m} b={bx},{bw}")
    x, w = rand((n, k), 1, torch.float32, dev).requires_grad_(), rand((m, k), 2, torch.float32, dev, 0.1).requires_grad_()
    dy = rand((n, m), 3, torch.float32, dev)
    y = quest_linear(x, w, block=block, bits_x=bx, bits_w=bw, compute_dtype=torch.float32, int8=True)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    q = []
    for t, bits in ((x, bx), (w, bw)):
        c, s, mask = qa.quantize_fwd_i8(t.detach(), block, bits, trust=1.3 if bits == 1 else 1.0, with_mask=True)
        v = mo.values(c.cpu().numpy().astype(np.float64), s.cpu().numpy(), bits)
        q.append((v, qo.unpack_lsb_first(mask.cpu().numpy(), 1, k).astype(np.float64)))
    (qx, mx), (qw, mw) = q
    want = qx @ qw.T
    # (the 64-bit sum of k rounded products is itself off by up to k + 2 half steps of the terms' sum: where the exact
    # sum is zero, the layer gives zero and this one a remainder)
    own = (np.abs(qx) @ np.abs(qw).T) * (k + 2) * 2.0 ** -53
    assert (np.abs(y.detach().double().cpu().numpy() - want) <= np.abs(want) * 8 * mo.U + own).all()
    d = dy.double().cpu().numpy()
    # a gradient: an fp32 product of values rounded to fp32 (3 roundings a term, one an addition), the transform
    # (log2(block) additions, one scaling)
    for got, g, terms, mask, count in ((dx, d @ qw, np.abs(d) @ np.abs(qw), mx, m), (dw, d.T @ qx, np.abs(d.T) @ np.abs(qx), mw, n)):
        bound = np.repeat((terms * (count + 4) * mo.U * mask).reshape(got.shape[0], -1, block).sum(-1) / block ** 0.5, block, 1)
        bound += np.repeat((np.abs(g) * mask).reshape(got.shape[0], -1, block).sum(-1) / block ** 0.5, block, 1) * (
            np.log2(block) + 3) * mo.U
        err = np.abs(got.double().cpu().numpy() - hadamard(g * mask, block))
        assert (err <= bound + 1e-30).all(), f"{(err / bound).max():.3g} of the bound"


def test_linear_follows_the_default_layer(dev):
    """bf16: as near to the 64-bit product as its output's rounding; the default layer rounds both operands first."""
    x, w = rand((64, 1024), 4, torch.bfloat16, dev), rand((200, 1024), 5, torch.bfloat16, dev, 0.05)
    y8 = quest_linear(x, w, bits_x=8, bits_w=8, int8=True)
    y = quest_linear(x, w, bits_x=8, bits_w=8)
    exact = quest_linear(x, w, bits_x=8, bits_w=8, compute_dtype=torch.float32, int8=True)
    assert torch.equal(y8, exact.to(torch.bfloat16))
    assert float((y.float() - exact).norm() / exact.norm()) < 3 * 2.0 ** -8


def test_linear_module(dev):
    log("module, bias, three axes, views, frozen")
    layer = QuestLinear(256, 96, bits_x=8, bits_w=8, int8=True, device=dev)
    with torch.no_grad():
        layer.bias.copy_(rand((96,), 6, torch.float32, dev))
    wide = rand((3, 7, 512), 7, torch.bfloat16, dev)
    x = wide[..., 1:257].detach().requires_grad_()  # neither contiguous nor aligned
    y = layer(x)
    assert y.shape == (3, 7, 96) and y.dtype == torch.bfloat16
    y.float().square().mean().backward()
    assert x.grad.shape == x.shape and all(torch.isfinite(p.grad).all() for p in layer.parameters())
    with torch.no_grad():
        want = layer(x)
    layer.freeze()
    assert layer._w_operand.dtype == torch.int8 and torch.equal(layer(x), want) and not layer(x).requires_grad is None
    with torch.no_grad():
        layer.weight.mul_(2.0)
    assert torch.equal(layer(x).detach(), want)  # the frozen weight
    layer.load_state_dict({k: v.clone() for k, v in layer.state_dict().items()})
    assert layer._w_operand is None and not torch.equal(layer(x).detach(), want)
    layer.freeze()
    layer.to(dev)
    assert layer._w_operand is None
    layer.freeze()
    layer.train()
    assert layer._w_operand is None


@pytest.mark.parametrize("need", [(True, False), (False, True)])
def test_linear_one_gradient(dev, need):
    x, w = rand((6, 128), 8, torch.bfloat16, dev), rand((10, 128), 9, torch.float32, dev)
    x.requires_grad_(need[0])
    w.requires_grad_(need[1])
    quest_linear(x, w, bits_x=8, bits_w=6, int8=True).float().sum().backward()
    assert (x.grad is not None) == need[0] and (w.grad is not None) == need[1]
    assert quest_linear(x[:0], w, bits_x=8, bits_w=8, int8=True).shape == (0, 10)


# ---------------------------------------------------------------------------
# The experts
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,bits_w,over_all", [(1, 4, False), (7, 4, True), (40, 8, False), (150, 4, False), (65, 6, False)])
def test_experts_frozen(dev, n, bits_w, over_all):
    """Frozen, the layer gives the definition's values of its own codes; unfrozen in fp32, nearly the same."""
    log(f"experts, {n} tokens, {bits_w} bits")
    moe = QuestMoE(256, 128, 12, 3, block=64, bits_x=8, bits_w=bits_w, compute_dtype=torch.float32, over_all=over_all, device=dev)
    x = rand((n, 256), 10, torch.bfloat16, dev)
    with torch.no_grad():
        plain = moe(x)
    moe.freeze()
    y = moe(x)
    assert y.shape == x.shape and y.dtype == torch.float32 and not y.requires_grad
    c, s, _ = qa.quantize_fwd_i8(x, 64, 8)
    values = []
    for codes, scale in zip(moe._frozen[::2], moe._frozen[1::2]):
        codes = codes.cpu().numpy()
        if bits_w == 4:
            codes = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.int64) - 8
        values.append(mo.values(codes.astype(np.float64), scale.cpu().numpy(), bits_w))
    logits = torch.nn.functional.linear(x.float(), moe.router)
    want, bound = mo.moe(mo.values(c.cpu().numpy().astype(np.float64), s.cpu().numpy(), 8), logits.double().detach().cpu().numpy(),
                         *values, 3, 64, 8, "silu", over_all)
    mo.check(y.double().cpu().numpy(), mo.U, want, bound)
    # unfrozen: the same codes but for a few at a level's edge, of h and of the weights
    assert float((plain - y).norm() / y.norm()) < 0.02
    assert torch.equal(moe(x.reshape(1, n, 256))[0], y)


def test_experts_train_a_step(dev):
    log("gradients and an optimizer step")
    moe = QuestMoE(128, 128, 4, 2, bits_x=8, bits_w=8, act="gelu", device=dev)
    opt = torch.optim.SGD(moe.parameters(), lr=1e-2)
    before = [p.detach().clone() for p in moe.parameters()]
    x = rand((2, 33, 128), 11, torch.bfloat16, dev).requires_grad_()
    moe(x).float().square().mean().backward()
    assert x.grad.shape == x.shape and all(torch.isfinite(p.grad).all() for p in moe.parameters())
    opt.step()
    assert all(not torch.equal(p, q) for p, q in zip(moe.parameters(), before))
    moe.freeze()
    assert moe._frozen is not None
    moe.train()
    assert moe._frozen is None


def test_router_gradient(dev):
    """The weights' gradient against differences, in 64 bits."""
    logits = rand((5, 9), 12, torch.float64, dev).requires_grad_()
    c = rand((5, 3), 13, torch.float64, dev)
    for over_all in (False, True):
        f = lambda l: (route(l, 3, over_all)[0].double() * c).sum()  # noqa: E731
        g = torch.autograd.grad(f(logits), logits)[0]
        for i, j in ((0, 0), (2, 5), (4, 8), (1, 3), (3, 7)):
            d = torch.zeros_like(logits)
            d[i, j] = 2.0 ** -6
            if not torch.equal(route(logits + d, 3)[1], route(logits - d, 3)[1]):
                assert (i, j) == (0, 0)  # other experts on either side of the logit: no derivative over the step
                continue
            slope = (f(logits + d) - f(logits - d)) / 2.0 ** -5
            # fp32 values of about 1 over a step of 2^-5, and a third derivative below 1
            assert abs(float((slope - g[i, j]).detach())) < 2.0 ** -15


# ---------------------------------------------------------------------------
# Together: a decoder layer's serving step, streams and graphs
# ---------------------------------------------------------------------------

def decoder_step(dev, n):
    """Norm, 8-bit projection, norm, experts: a frozen layer without its attention, and its pieces."""
    proj = QuestLinear(256, 256, bias=False, bits_x=8, bits_w=8, int8=True, device=dev).freeze()
    moe = QuestMoE(256, 128, 16, 2, bits_x=8, device=dev).freeze()

    def step(x):
        with torch.no_grad():
            x = x + proj(layer_norm(x))
            return x + moe(layer_norm(x))

    return step, [rand((n, 256), 20 + i, torch.bfloat16, dev) for i in range(2)]


@pytest.mark.parametrize("n", [1, 5, 48])
def test_layer_in_graphs(dev, n):
    """Two captured graphs of the step, replayed in turn with eager work between: every replay gives the eager bits."""
    log(f"graphs, {n} tokens")
    step, xs = decoder_step(dev, n)
    want = [step(x) for x in xs]
    graphs = []
    for x in xs:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(x)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(x)
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), ref in zip(graphs, want):
            out.fill_(3.0)
            torch.cuda.synchronize()
            g.replay()
            again = step(xs[0])
            torch.cuda.synchronize()
            assert torch.equal(out, ref) and torch.equal(again, want[0])


def test_training_step_in_a_graph(dev):
    """The 8-bit linear layer's forward and backward captured and replayed."""
    x, w = rand((40, 256), 30, torch.bfloat16, dev), rand((96, 256), 31, torch.bfloat16, dev)
    dy = rand((40, 96), 32, torch.bfloat16, dev)

    def step():
        a, b = x.detach().requires_grad_(), w.detach().requires_grad_()
        y = quest_linear(a, b, bits_x=8, bits_w=8, int8=True)
        return (y.detach(), *torch.autograd.grad(y, (a, b), dy))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for _ in range(3):
        for o in outs:
            o.fill_(2.0)
        torch.cuda.synchronize()
        g.replay()
        again = step()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, want)) and all(torch.equal(o, r) for o, r in zip(again, want))


def test_two_streams_at_once(dev):
    """The same layer on two streams at a time, and calls given a stream."""
    step, xs = decoder_step(dev, 40)
    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(xs[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    c, s, _ = qa.quantize_fwd_i8(xs[0], 128, 8)
    w, ws, _ = qa.quantize_fwd_i8(xs[1], 128, 8)
    ref = qa.gemm_i8(c, s, 8, w, ws, 8), qa.dequantize_i8(c, s, 8)
    streams[0].wait_stream(torch.cuda.current_stream())
    c2, s2, _ = qa.quantize_fwd_i8(xs[0], 128, 8, stream=streams[0])
    y2 = qa.gemm_i8(c2, s2, 8, w, ws, 8, stream=streams[0])
    v2 = qa.dequantize_i8(c2, s2, 8, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(y2, ref[0]) and torch.equal(v2, ref[1])


def test_frozen_product_call(dev):
    x, w = rand((3, 4, 256), 40, torch.float32, dev), rand((72, 256), 41, torch.float32, dev)
    codes, scale, _ = qa.quantize_fwd_i8(w, 64, 5)
    y = quest_linear_int8(x, codes, scale, 5, bias=torch.ones(72, device=dev), block=64, bits_x=7, out_dtype=torch.float32)
    cx, sx, _ = qa.quantize_fwd_i8(x.reshape(12, 256), 64, 7)
    assert torch.equal(y.reshape(12, 72), qa.gemm_i8(cx, sx, 7, codes, scale, 5, out_dtype=torch.float32) + 1.0)


@pytest.mark.parametrize("x_dtype,w_dtype,compute", [
    (torch.bfloat16, torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32, torch.bfloat16),
    (torch.float32, torch.bfloat16, torch.float32), (torch.float32, torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("n,bits_w", [(64, 8), (7, 6), (0, 8)])
def test_gradients_of_each_type(dev, x_dtype, w_dtype, compute, n, bits_w):
    """Gradients come in their tensors' types, those in fp32 without a rounding to bf16 on the way."""
    log(f"gradient types n={n} bits {bits_w} {x_dtype} {w_dtype} {compute}")
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(n, 256, generator=gen).to(dev, x_dtype).requires_grad_()
    w = torch.randn(96, 256, generator=gen).to(dev, w_dtype).requires_grad_()
    dy = torch.randn(n, 96, generator=gen).to(dev, compute)
    y = quest_linear(x, w, bits_x=8, bits_w=bits_w, compute_dtype=compute, int8=True)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert dx.dtype == x_dtype and dw.dtype == w_dtype and dx.shape == x.shape and dw.shape == w.shape
    if not n:
        assert (dw == 0).all()
        return
    qs = []
    for t, b in ((x, 8), (w, bits_w)):
        c, s, m = qa.quantize_fwd_i8(t.detach(), 128, b, with_mask=True)
        qs.append((qa.dequantize_i8(c, s, b, out_dtype=compute).double(), m))
    # In 64 bits from the values that are multiplied; the products' fp32 sums of n or 96 terms and the transform's
    # seven additions and factor are off by at most so many steps of the sum of magnitudes.
    for got, g, size, m in ((dx, dy.double() @ qs[1][0], dy.double().abs() @ qs[1][0].abs(), qs[0][1]),
                            (dw, dy.double().t() @ qs[0][0], dy.double().abs().t() @ qs[0][0].abs(), qs[1][1])):
        shifts = torch.arange(8, dtype=torch.uint8, device=dev)
        keep = ((m.reshape(-1, 1) >> shifts) & 1).reshape(g.shape).double()
        had = torch.ones(1, 1, dtype=torch.float64, device=dev)
        while len(had) < 128:
            had = torch.cat([torch.cat([had, had], 1), torch.cat([had, -had], 1)])
        want = ((g * keep).reshape(-1, 128) @ had / 128 ** 0.5).reshape(g.shape)
        most = (size.reshape(-1, 128).sum(-1, keepdim=True) / 128 ** 0.5).expand(-1, 128).reshape(g.shape)
        eps = torch.finfo(got.dtype).eps / 2
        assert ((got.double() - want).abs() <= eps * want.abs() + (max(n, 96) + 9) * 2.0 ** -24 * most * (1 + eps)).all()


def test_no_tokens(dev):
    layer = QuestMoE(128, 128, 4, 2, device=dev, dtype=torch.bfloat16)
    assert layer(torch.zeros(0, 128, dtype=torch.bfloat16, device=dev)).shape == (0, 128)
    assert layer.freeze()(torch.zeros(2, 0, 128, dtype=torch.bfloat16, device=dev)).shape == (2, 0, 128)
