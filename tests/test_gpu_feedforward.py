"""The feed-forward block's modules: gradients against the definitions in 64 bits, the whole block as it is used,
its frozen form, and its calls in HIP graphs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import feedforward_oracle as fo
import quantization_aware_amd as qa
from oracle import quest_oracle as qo
from quantization_aware_amd.feedforward import LayerNorm, QuestFeedForward, layer_norm, quest_gated
from quantization_aware_amd.linear import quest_linear

pytestmark = pytest.mark.gpu


def log(msg: str) -> None:
    print(f"[gpu-ff] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    return torch.device("cuda", 0)


def rand(shape, seed, dtype, dev, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=g)).to(dtype).to(dev)


# ---------------------------------------------------------------------------
# Layer norm under autograd
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("shape,pdtype", [((3, 5, 384), torch.float32), ((2, 1001), torch.bfloat16), ((64,), torch.float32)])
def test_layer_norm_gradients(dev, shape, pdtype, act8):
    log(f"layer_norm {shape} {pdtype} act8={act8}")
    cols = shape[-1]
    x = rand(shape, 1, torch.float32, dev).requires_grad_()
    w = (1 + rand((cols,), 2, torch.float32, dev, 0.2)).to(pdtype).requires_grad_()
    b = rand((cols,), 3, pdtype, dev, 0.2).requires_grad_()
    dy = rand(shape, 4, torch.float32, dev, 1e-2)
    y = layer_norm(x, w, b, act8=act8)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    x2, dy2 = x.detach().reshape(-1, cols), dy.reshape(-1, cols)
    wy, wm, wr, wx = fo.norm_fwd(fo.f64(x2), fo.f64(w), fo.f64(b), 1e-5)
    ey, _, er, ex = fo.norm_fwd_bounds(fo.f64(x2), fo.f64(w), fo.f64(b), 1e-5)
    fo.check("y", y.reshape(-1, cols), wy, ey)
    # the calls that the function stands for
    yk, mean, rstd, kept = qa.layer_norm_fwd(x2, w.detach(), b.detach(), act8=act8)
    src = dict(act8=kept) if act8 else dict(x=x2, mean=mean)
    want = qa.layer_norm_bwd(dy2, rstd, w.detach(), bias_grad=True, **src)
    assert torch.equal(dx.reshape(-1, cols), want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])
    assert dw.dtype == pdtype


def test_layer_norm_partial_gradients_and_views(dev):
    log("frozen parameters, a misaligned view of x, no gradient")
    base = rand((7, 641), 5, torch.bfloat16, dev)
    x = base[:, 1:]  # neither contiguous nor aligned
    norm = LayerNorm(640, device=dev)
    norm.weight.requires_grad_(False)
    leaf = x.clone().requires_grad_()
    y = norm(leaf)
    y.sum().backward()
    assert norm.weight.grad is None and norm.bias.grad is not None and leaf.grad is not None
    with torch.no_grad():
        assert torch.equal(norm(x), y)
    flat = base.flatten()[1:1 + 640].unsqueeze(0)  # contiguous, 2 bytes past a 16-byte boundary
    assert torch.equal(layer_norm(flat), layer_norm(flat.clone()))


def test_layer_norm_expanded_gradient(dev):
    log("broadcast dy and x")
    x = rand((1, 96), 6, torch.float32, dev).requires_grad_()
    y = layer_norm(x.expand(10, 96))
    y.sum().backward()
    x2 = x.detach().clone().requires_grad_()
    layer_norm(x2).backward(torch.full((1, 96), 10.0, device=dev))
    # ten equal rows added by torch: 10 roundings of each term
    assert torch.allclose(x.grad, x2.grad, rtol=0, atol=float(20 * fo.U * 10 * 96 ** 0.5))


# ---------------------------------------------------------------------------
# The gated product under autograd
# ---------------------------------------------------------------------------

def reference_gradients(dev, x, gate, up, dh, block, bx, bw, act, trust_x, trust_w, cd):
    """(dx, dgate, dup) and their bounds: from the codes and masks that the quantiser gives and the 8-bit
    checkpoints of the products, in 64 bits, with the roundings of the block's own steps counted."""
    n, k = x.shape
    m = gate.shape[0]
    cx, sx, mx, ox = qa.quantize_fwd_op(x, block, bx, trust=trust_x, with_codes=True, with_mask=True)
    lev, masks, kept = [], [], []
    for w in (gate, up):
        c, s, mk, o = qa.quantize_fwd_op(w, block, bw, trust=trust_w, with_codes=True, with_mask=True)
        lev.append(fo.f64(qa.dequantize(c, s, m, k, bw, out_dtype=cd)))
        masks.append(mk.cpu().numpy())
        codes, scale = qa.act8_save(qa.gemm(ox, sx, n, bx, o, s, m, bw, k, out_dtype=torch.float32))
        kept.append(fo.act8_values(codes.cpu().numpy(), scale.cpu().numpy()))
    qx = fo.f64(qa.dequantize(cx, sx, n, k, bx, out_dtype=cd))
    qw = np.concatenate(lev)
    wmask = np.concatenate(masks)
    dgu, err = fo.gated_bwd(fo.f64(dh.to(cd)), kept[0], kept[1], act)
    hs = fo.half_step(cd)
    err = err + hs * (np.abs(dgu) + err)
    out = []
    for left, le, right, mask in ((dgu.T, err.T, qx, wmask), (dgu, err, qw, mx.cpu().numpy())):
        g = left @ right
        # the product's fp32 sum of its terms in any order, and its rounding to the compute type
        ge = le @ np.abs(right) + left.shape[1] * fo.U * (np.abs(left) @ np.abs(right))
        ge = ge + hs * (np.abs(g) + ge)
        want = qo.trust_bwd(g, mask, block)
        # an orthonormal transform: an entry's error is at most the block's 2-norm; its fp32 steps, the rounding
        rows, cols = g.shape
        norm = np.sqrt((ge ** 2).reshape(rows, -1, block).sum(-1, keepdims=True))
        size = np.sqrt((g ** 2).reshape(rows, -1, block).sum(-1, keepdims=True))
        we = np.broadcast_to(norm + 16 * fo.U * size + hs * 0, (rows, cols // block, block)).reshape(rows, cols)
        out.append((want, we))
    (dw, dwe), (dx, dxe) = out
    return (dx, dxe), (dw[:m], dwe[:m]), (dw[m:], dwe[m:])


@pytest.mark.parametrize("n,k,m,block,bx,bw,act,cd", [
    (64, 256, 96, 128, 4, 4, "silu", torch.bfloat16),
    (33, 384, 130, 64, 4, 4, "gelu", torch.float32),
    (7, 128, 41, 128, 2, 3, "silu", torch.float32),
    (130, 512, 64, 256, 1, 1, "silu", torch.bfloat16),
])
def test_gated_gradients(dev, n, k, m, block, bx, bw, act, cd):
    log(f"quest_gated {n}x{k}x{m} block {block} b={bx},{bw} {act} {cd}")
    x = rand((n, k), 11, torch.bfloat16, dev).requires_grad_()
    gate = rand((m, k), 12, torch.bfloat16, dev, k ** -0.5).requires_grad_()
    up = rand((m, k), 13, torch.bfloat16, dev, k ** -0.5).requires_grad_()
    dh = rand((n, m), 14, torch.float32, dev, 1e-2)
    h = quest_gated(x, gate, up, block, bx, bw, cd, act)
    got = torch.autograd.grad(h, (x, gate, up), dh.to(cd))
    t = 1.3 if bx == 1 else 1.0, 1.3 if bw == 1 else 1.0
    refs = reference_gradients(dev, x.detach(), gate.detach(), up.detach(), dh, block, bx, bw, act, *t, cd)
    for name, g, (want, err) in zip(("dx", "dgate", "dup"), got, refs):
        # (for an fp32 compute type the gradient is rounded to the bf16 leaf at the end)
        r = fo.check(name, g, want, err)
        log(f"{name} error / tolerance {r:.3g}")
    # the parts of it: the same products as two quantised linear maps
    g2 = quest_linear(x.detach(), gate.detach(), None, block, bx, bw, torch.float32)
    u2 = quest_linear(x.detach(), up.detach(), None, block, bx, bw, torch.float32)
    hv, _, hb, _ = fo.act(fo.f64(g2), act)
    fo.check("h", h, hv * fo.f64(u2), np.abs(fo.f64(u2)) * hb + 2 * fo.U * np.abs(hv * fo.f64(u2)))


@pytest.mark.parametrize("n,k,m,block,bx,bw,act", [
    (64, 256, 96, 128, 4, 4, "silu"), (64, 256, 96, 128, 4, 4, "gelu"), (130, 512, 64, 256, 1, 1, "silu"),
    (300, 384, 260, 64, 2, 4, "gelu"),
])
def test_gated_gradients_of_jointly_kept_weights(dev, n, k, m, block, bx, bw, act):
    """Widths that are multiples of 4, whose two weights are rebuilt and masked as one: in fp32, entry by entry within
    the counted roundings; in bf16, as a whole within 2^-8 of each gradient's norm.  (Three roundings to bf16 stand
    behind an entry, of the product's left operand, its result and the output; each errs by 0.42 2^-8 of the value,
    rms, and independently, together 0.74 2^-8; the bytes behind both sides are the same.  The fp32 bound is 64 half
    steps, the same three and the products' sums of up to 520 terms.)"""
    log(f"quest_gated closely {n}x{k}x{m} block {block} b={bx},{bw} {act}")
    t = 1.3 if bx == 1 else 1.0, 1.3 if bw == 1 else 1.0
    for cd in (torch.float32, torch.bfloat16):
        x = rand((n, k), 11, cd, dev).requires_grad_()
        gate = rand((m, k), 12, cd, dev, k ** -0.5).requires_grad_()
        up = rand((m, k), 13, cd, dev, k ** -0.5).requires_grad_()
        dh = rand((n, m), 14, cd, dev, 1e-2)
        got = torch.autograd.grad(quest_gated(x, gate, up, block, bx, bw, cd, act), (x, gate, up), dh)
        refs = reference_gradients(dev, x.detach(), gate.detach(), up.detach(), dh, block, bx, bw, act, *t, cd)
        for name, g, (want, err) in zip(("dx", "dgate", "dup"), got, refs):
            off = np.linalg.norm(fo.f64(g) - want) / np.linalg.norm(want)
            log(f"{cd} {name}: {off * 256:.3g} 2^-8 of its norm")
            if cd == torch.float32:
                fo.check(name, g, want, err)
            assert off <= 2.0 ** (-8 if cd == torch.bfloat16 else -18), (name, off)


@pytest.mark.parametrize("needs", [(True, False, False), (False, True, False), (False, False, True), (False, True, True)])
def test_gated_partial_gradients(dev, needs):
    log(f"gradients of {needs}")
    ts = [rand((20, 256), 21, torch.float32, dev), rand((48, 256), 22, torch.float32, dev, 0.06),
          rand((48, 256), 23, torch.float32, dev, 0.06)]
    full = [t.clone().requires_grad_() for t in ts]
    part = [t.clone().requires_grad_(r) for t, r in zip(ts, needs)]
    for leaves in (full, part):
        quest_gated(*leaves).float().square().sum().backward()
    for f, p, r in zip(full, part, needs):
        assert (p.grad is None) == (not r)
        if r:
            assert torch.equal(f.grad, p.grad)


def test_gated_keeps_eight_bits(dev):
    """What autograd saves: codes and masks of the operands and 8.25 bits for each product's entry, once."""
    log("saved bytes")
    n, k, m = 512, 256, 1024
    x, gate, up = (rand(s, i, torch.bfloat16, dev).requires_grad_() for i, s in enumerate(((n, k), (m, k), (m, k))))
    seen = {}
    with torch.autograd.graph.saved_tensors_hooks(lambda t: seen.setdefault(t.data_ptr(), t), lambda t: t):
        quest_gated(x, gate, up)
    total = sum(t.numel() * t.element_size() for t in seen.values())
    operands = (n + 2 * m) * (k // 2 + k // 8 + 4)
    assert total == operands + 2 * n * m + 2 * n * m // 32


def test_gated_without_gradient_and_empty(dev):
    log("no gradient, no rows")
    x, gate, up = (rand(s, i, torch.bfloat16, dev) for i, s in enumerate(((2, 3, 256), (72, 256), (72, 256))))
    h = quest_gated(x, gate, up)
    assert h.shape == (2, 3, 72) and not h.requires_grad
    h2 = quest_gated(x.requires_grad_(), gate, up)
    assert torch.equal(h, h2)
    gate.requires_grad_()
    h = quest_gated(x[:0], gate, up)
    h.sum().backward()
    assert h.shape == (0, 3, 72) and not gate.grad.any()


def test_no_checkpoint_without_a_gradient(dev):
    """Under no_grad nothing is kept, whatever the parameters require."""
    log("no_grad allocates no checkpoint")
    x, gate, up = (rand(s, i, torch.bfloat16, dev).requires_grad_() for i, s in
                   enumerate(((4096, 128), (8192, 128), (8192, 128))))
    quest_gated(x[:1], gate, up)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with torch.no_grad():
        h = quest_gated(x, gate, up)
    # h, the three operands and scales; the checkpoints would be two more bytes an entry of h
    assert torch.cuda.max_memory_allocated() - before < 1.5 * h.numel() * 2


def test_calls_on_their_own_stream(dev):
    """A call given a stream takes its memory there: blocks that the current stream is still writing are not
    among its outputs or its workspace."""
    log("memory of a call on another stream")
    rows, cols = 4096, 2048
    x, dy = rand((rows, cols), 1, torch.bfloat16, dev), rand((rows, cols), 2, torch.bfloat16, dev)
    w = rand((cols,), 3, torch.float32, dev)
    y, mean, rstd, kept = qa.layer_norm_fwd(x, w, w, act8=True)
    want = qa.layer_norm_bwd(dy, rstd, w, act8=kept, bias_grad=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        # freed blocks of the sizes the call needs, which the current stream writes for a while yet
        junk = [torch.empty_like(x) for _ in range(2)] + [torch.empty(512 * 2 * cols, device=dev)]
        for _ in range(20):
            for j in junk:
                j.fill_(7.0)
        del junk
        got = qa.layer_norm_bwd(dy, rstd, w, act8=kept, bias_grad=True, stream=side)
        torch.cuda.synchronize()
        for a, c in zip(got, want):
            assert torch.equal(a, c)


def test_two_streams_at_once(dev):
    """The same calls in flight on two streams: each has its own workspace and outputs."""
    log("two streams")
    sets = []
    for i in range(2):
        x, dy = rand((3000, 1024), 40 + i, torch.bfloat16, dev), rand((3000, 1024), 50 + i, torch.bfloat16, dev)
        w = rand((1024,), 60 + i, torch.float32, dev)
        ops = [qa.quantize_fwd_op(rand((r, 1024), 70 + i, torch.bfloat16, dev), 128, 4) for r in (1024, 1024)]
        sets.append((x, dy, w, ops))

    def work(x, dy, w, ops, stream=None):
        y, _, rstd, kept = qa.layer_norm_fwd(x, w, w, act8=True, stream=stream)
        _, xs, _, xo = qa.quantize_fwd_op(x, 128, 4)
        h, g8, u8 = qa.gated_fwd(xo, xs, 3000, 4, ops[0][3], ops[0][1], ops[1][3], ops[1][1], 1024, 4, 1024, act8=True,
                                 stream=stream)
        return (y, h, qa.gated_bwd(h, g8, u8, stream=stream),
                *qa.layer_norm_bwd(dy, rstd, w, act8=kept, bias_grad=True, stream=stream))

    want = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(work(*s, stream=st))
        torch.cuda.synchronize()
        for g, r in zip(got, want):
            assert all(torch.equal(a, c) for a, c in zip(g, r))


def test_gated_refusals(dev):
    log("refusals")
    x, w = rand((4, 256), 1, torch.bfloat16, dev), rand((8, 256), 2, torch.bfloat16, dev)
    for kw, exc in ((dict(bits_x=5), ValueError), (dict(act="relu"), ValueError), (dict(block=96), ValueError),
                    (dict(compute_dtype=torch.float16), TypeError)):
        with pytest.raises(exc):
            quest_gated(x, w, w, **kw)
    with pytest.raises(ValueError):
        quest_gated(x, w, w[:4])
    with pytest.raises(ValueError):
        quest_gated(x[:, :192], w[:, :192], w[:, :192])
    with pytest.raises(TypeError):
        quest_gated(x.half(), w, w)


# ---------------------------------------------------------------------------
# The block
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("norm", [True, False])
def test_block_is_its_parts(dev, norm):
    """A training step of the block equals the same step through its public parts, bit for bit."""
    log(f"block, norm={norm}")
    torch.manual_seed(5)
    ff = QuestFeedForward(256, 384, norm=norm, device=dev)
    if norm:
        with torch.no_grad():
            ff.norm.weight.add_(rand((256,), 3, torch.float32, dev, 0.1))
            ff.norm.bias.add_(rand((256,), 4, torch.float32, dev, 0.1))
    x = rand((3, 40, 256), 6, torch.bfloat16, dev).requires_grad_()
    dout = rand((3, 40, 256), 7, torch.bfloat16, dev, 1e-2)
    out = ff(x)
    out.backward(dout)
    grads = [p.grad.clone() for p in ff.parameters()] + [x.grad.clone()]
    assert all(torch.isfinite(g).all() and g.any() for g in grads)
    for p in ff.parameters():
        p.grad = None
    x2 = x.detach().clone().requires_grad_()
    y = layer_norm(x2, ff.norm.weight, ff.norm.bias, act8=True) if norm else x2
    h = quest_gated(y, ff.gate, ff.up)
    out2 = quest_linear(h, ff.down.weight)
    out2.backward(dout)
    assert torch.equal(out, out2)
    for a, c in zip(grads, [p.grad for p in ff.parameters()] + [x2.grad]):
        assert torch.equal(a, c)


def test_block_trains_a_step(dev):
    log("optimizer step")
    ff = QuestFeedForward(128, 256, device=dev)
    opt = torch.optim.SGD(ff.parameters(), lr=1e-2)
    before = [p.detach().clone() for p in ff.parameters()]
    for i in range(3):
        opt.zero_grad()
        ff(rand((64, 128), 30 + i, torch.bfloat16, dev)).float().square().mean().backward()
        opt.step()
    assert all(torch.isfinite(p).all() and not torch.equal(p, q) for p, q in zip(ff.parameters(), before))


@pytest.mark.parametrize("tokens", [1, 5, 200])
def test_frozen_block(dev, tokens):
    """Frozen, the block gives what it gives unfrozen without gradients; training, loading and moving thaw it."""
    log(f"frozen, {tokens} tokens")
    ff = QuestFeedForward(256, 384, act="gelu", device=dev)
    x = rand((tokens, 256), 8, torch.bfloat16, dev)
    with torch.no_grad():
        want = ff(x)
    ff.freeze()
    assert not ff.training and torch.equal(ff(x), want)
    with torch.no_grad():
        ff.gate.mul_(2.0)
    assert torch.equal(ff(x), want)  # the frozen weights
    ff.train()
    assert ff._frozen is None and ff.down._w_operand is None
    changed = ff(x).detach()
    assert not torch.equal(changed, want)
    ff.freeze()
    state = {k: v.clone() for k, v in ff.state_dict().items()}
    state["gate"] /= 2.0
    ff.load_state_dict(state)
    assert ff._frozen is None and torch.equal(ff(x).detach(), want)
    ff.freeze()
    ff.to(dev)
    assert ff._frozen is None


def test_block_one_bit(dev):
    log("one bit")
    ff = QuestFeedForward(128, 128, bits_x=1, bits_w=1, device=dev)
    assert ff.trust_x == 1.3
    ff(rand((9, 128), 8, torch.float32, dev)).sum().backward()
    assert all(torch.isfinite(p.grad).all() for p in ff.parameters())


# ---------------------------------------------------------------------------
# HIP graphs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,k,m", [(300, 512, 384), (3, 256, 200), (129, 128, 41)])
def test_step_in_graphs(dev, n, k, m):
    """The operators' step captured twice, both graphs replayed in turn with eager work between: each replay
    gives the eager bits (nothing is kept between calls, and the graphs share no workspace)."""
    log(f"graphs of {n}x{k}x{m}")
    x, dy = rand((n, k), 1, torch.bfloat16, dev), rand((n, k), 2, torch.bfloat16, dev)
    w, b = rand((k,), 3, torch.float32, dev), rand((k,), 4, torch.float32, dev)
    dh = rand((n, m), 5, torch.bfloat16, dev)
    ops = [qa.quantize_fwd_op(rand((r, k), 6 + r, torch.bfloat16, dev), 128, 4) for r in (m, m)]

    def step(src):
        y, _, rstd, kept = qa.layer_norm_fwd(src, w, b, act8=True)
        _, xs, _, xo = qa.quantize_fwd_op(y, 128, 4)
        h, g8, u8 = qa.gated_fwd(xo, xs, n, 4, ops[0][3], ops[0][1], ops[1][3], ops[1][1], m, 4, k, act8=True)
        dgu = qa.gated_bwd(dh, g8, u8)
        back = qa.act8_load(*qa.act8_save(h))
        return (y, h, dgu, back, *qa.layer_norm_bwd(dy, rstd, w, act8=kept, bias_grad=True))

    srcs = [x, x.flip(0).contiguous()]
    want = [step(s) for s in srcs]
    torch.cuda.synchronize()
    graphs = []
    for s in srcs:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(s)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(s)
        graphs.append((g, outs))
    for replay in range(3):
        for (g, outs), ref in zip(graphs, want):
            for o in outs:
                o.fill_(3.0)
            torch.cuda.synchronize()
            g.replay()
            again = step(srcs[0])  # eager calls behind the replay
            torch.cuda.synchronize()
            for i, (o, r) in enumerate(zip(outs, ref)):
                assert torch.equal(o, r), f"replay {replay}, output {i}"
            assert all(torch.equal(p, q) for p, q in zip(again, want[0]))
