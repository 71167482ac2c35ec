"""The feed-forward half of a decoder layer around the quantised products.

    y = norm(x),  h = act(Q(y) Q(gate)^T) * (Q(y) Q(up)^T),  out = Q(h) Q(down)^T

Layer norm (quest_layer_norm_fwd / _bwd), the gated product of quantised
operands (quest_gated_fwd / _bwd) and QuestLinear's product, with the
quantiser of QuestLinear on every operand (the pages quantise the inputs and
weights of every linear layer: pith.science review of QuEST, "What carries
the argument").

What the backward pass keeps.  The gated product saves the 4-bit codes and
trust masks of its operands, as QuestLinear does, and its two products, which
the activation's gradient needs, in 8 bits (8.25 with the exponents, against
16 in bf16 or 32): the gradients are those of act(g) u at the saved values
(each within 2^-7 of the largest of its block of 32, 2^-6 where it is that
largest).  Against gradients at the unrounded products, dx, dgate and dup of
normal activations by normal weights (4096 x 2048 -> 5632) are off by 0.8 to 1.3%
of their norm, where products kept in bf16 give 0.2%.  Layer norm can keep its
normalised input the same way (``act8``).
As in QuestLinear, the products of the backward pass are plain library GEMMs
through torch on the dequantised operands; both weights' gradients are one of
them and one trust backward, and so is the input's.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (ACTIVATIONS, dequantize, gated_bwd, gated_fwd, layer_norm_bwd, layer_norm_fwd, quantize_fwd_op,
               quantize_fwd_op_group, trust_bwd)
from .linear import QuestLinear, _dense, default_trust

__all__ = ["layer_norm", "LayerNorm", "quest_gated", "QuestFeedForward"]


def _differentiates(*tensors) -> bool:
    """Whether a backward pass can follow (inside a Function's forward, torch.is_grad_enabled() no longer tells)."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


class LayerNormFunction(torch.autograd.Function):
    """Layer norm of the rows of a 2-D x; see layer_norm."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, act8):
        y, mean, rstd, kept = layer_norm_fwd(x, weight, bias, eps, act8=act8)
        ctx.act8 = act8
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.save_for_backward(weight, rstd, *(kept if act8 else (x, mean)))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weight, rstd, a, b = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        src = dict(act8=(a, b)) if ctx.act8 else dict(x=a, mean=b)
        dx, dw, db = layer_norm_bwd(_dense(dy), rstd, weight, input_grad=need_x, weight_grad=need_w, bias_grad=need_b,
                                    param_dtype=ctx.bias_dtype, **src)
        return dx, dw, db, None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5, act8: bool = False) -> torch.Tensor:
    """Layer norm over the last axis of x (float32 or bfloat16), differentiable.

    weight, bias: (cols,) of one type, float32 or bfloat16, or None.  act8:
    keep the normalised input in 8 bits for the backward pass instead of x.
    """
    flat = _dense(x.reshape(-1, x.shape[-1]))
    weight, bias = (None if t is None else _dense(t) for t in (weight, bias))
    return LayerNormFunction.apply(flat, weight, bias, eps, act8 and _differentiates(flat, weight, bias)).reshape(x.shape)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last axis, of `features` entries; act8 as in layer_norm."""

    def __init__(self, features: int, eps: float = 1e-5, weight: bool = True, bias: bool = True, act8: bool = False,
                 device=None, dtype=None):
        super().__init__()
        self.eps, self.act8 = eps, act8
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype)) if weight else None
        self.bias = torch.nn.Parameter(torch.zeros(features, device=device, dtype=dtype)) if bias else None
        self.features = features

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.features:
            raise ValueError(f"the last axis of x has {x.shape[-1]} entries, the norm {self.features}")
        return layer_norm(x, self.weight, self.bias, self.eps, self.act8)


def _quantise_operands(x, gate, up, block, bits_x, bits_w, trust_x, trust_w, keep: bool):
    """Operands and scales of x, gate and up and, with keep, what the backward pass needs of them.

    Returns ((operand, scale) of each, saved): saved is (codes, scale, mask) of
    x and of both weights, those of the weights as rows of one tensor (gate's,
    then up's), so that one launch rebuilds, and one masks, both.  The up half's
    scales start on a 16-byte boundary, behind up to 3 unused ones.
    """
    dev, k = x.device, x.shape[1]

    def buffers(rows, bits):
        return (torch.empty((rows, k * bits // 8), dtype=torch.uint8, device=dev),
                torch.empty((rows, k // 8), dtype=torch.uint8, device=dev))

    m = gate.shape[0]
    second = -(-m // 4) * 4
    w_scale = torch.empty((second + m,), dtype=torch.float32, device=dev)
    outs = [{}, dict(scale=w_scale[:m]), dict(scale=w_scale[second:])]
    saved = ()
    if keep:
        xc, xm = buffers(x.shape[0], bits_x)
        wc, wm = buffers(2 * m, bits_w)
        outs[0].update(codes=xc, mask=xm)
        outs[1].update(codes=wc[:m], mask=wm[:m])
        outs[2].update(codes=wc[m:], mask=wm[m:])
    same = bits_x == bits_w and trust_x == trust_w and x.dtype == gate.dtype == up.dtype
    if same:
        got = quantize_fwd_op_group([x, gate, up], block, bits_x, trust=trust_x, outs=outs)
    else:
        got = [quantize_fwd_op(x, block, bits_x, trust=trust_x, **outs[0])]
        got += [quantize_fwd_op(w, block, bits_w, trust=trust_w, **o) for w, o in ((gate, outs[1]), (up, outs[2]))]
    if keep:
        saved = (xc, got[0][1], xm, wc, w_scale, wm)
    return [(op, scale) for _, scale, _, op in got], saved


class QuestGatedFunction(torch.autograd.Function):
    """h = act(Q(x) Q(gate)^T) * (Q(x) Q(up)^T) for 2-D x; see quest_gated."""

    @staticmethod
    def forward(ctx, x, gate, up, block, bits_x, bits_w, compute_dtype, act, trust_x, trust_w, keep):
        ops, saved = _quantise_operands(x, gate, up, block, bits_x, bits_w, trust_x, trust_w, keep)
        (xo, xs), (go, gs), (uo, us) = ops
        (n, k), m = x.shape, gate.shape[0]
        h, gate8, up8 = gated_fwd(xo, xs, n, bits_x, go, gs, uo, us, m, bits_w, k, act=act, out_dtype=compute_dtype,
                                  act8=keep)
        if keep:
            ctx.save_for_backward(*saved, *gate8, *up8)
        ctx.dims = (n, m, k, block, bits_x, bits_w, compute_dtype, act)
        ctx.dtypes = (x.dtype, gate.dtype, up.dtype)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        xc, xs, xm, wc, ws, wm, gc, gs, uc, us = ctx.saved_tensors
        n, m, k, block, bits_x, bits_w, compute_dtype, act = ctx.dims
        need_x, need_g, need_u = ctx.needs_input_grad[:3]
        dgu = gated_bwd(_dense(dh.to(compute_dtype)), (gc, gs), (uc, us), act=act)  # [dg | du]
        dx = dg = du = None
        if need_g or need_u:
            # gradients reaching Q(gate) and Q(up), Hadamard domain, as rows of one product
            g = torch.mm(dgu.t(), dequantize(xc, xs, n, k, bits_x, out_dtype=compute_dtype))
            trust_bwd(g, wm, block, out=g)
            dg = g[:m].to(ctx.dtypes[1]) if need_g else None
            du = g[m:].to(ctx.dtypes[2]) if need_u else None
        if need_x:
            if m % 4 == 0:
                qw = dequantize(wc, ws, 2 * m, k, bits_w, out_dtype=compute_dtype)
            else:
                qw = torch.empty((2 * m, k), dtype=compute_dtype, device=dgu.device)
                dequantize(wc[:m], ws[:m], m, k, bits_w, out=qw[:m])
                dequantize(wc[m:], ws[-m:], m, k, bits_w, out=qw[m:])
            g = torch.mm(dgu, qw)  # gradient reaching Q(x)
            dx = trust_bwd(g, xm, block, out=g).to(ctx.dtypes[0])
        return dx, dg, du, None, None, None, None, None, None, None, None


def _check_gated(in_features: int, block: int, bits_x: int, bits_w: int, act: str, compute_dtype) -> None:
    if not (1 <= bits_x <= 4 and 1 <= bits_w <= 4):
        raise ValueError(f"the gated product takes operands of 1 to 4 bits, not {bits_x} and {bits_w}")
    if in_features % 128 or in_features % block:
        raise ValueError(f"in_features ({in_features}) must be a multiple of 128 and of the Hadamard block ({block})")
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {tuple(ACTIVATIONS)}, not {act!r}")
    if compute_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"compute_dtype is float32 or bfloat16, not {compute_dtype}")


def quest_gated(x: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, block: int = 128, bits_x: int = 4,
                bits_w: int = 4, compute_dtype=torch.bfloat16, act: str = "silu", trust_x: float | None = None,
                trust_w: float | None = None) -> torch.Tensor:
    """act(Q(x) Q(gate)^T) * (Q(x) Q(up)^T) of x (..., K) by gate and up (M, K), differentiable.

    On the "int" grid, with the trust factors of quest_linear; K a multiple of
    128 and of block.  act: "silu" or "gelu" (with the normal distribution
    function).
    """
    if x.shape[-1] != gate.shape[-1] or gate.shape != up.shape or gate.dim() != 2:
        raise ValueError(f"x (..., K) by gate and up (M, K): got {tuple(x.shape)}, {tuple(gate.shape)} and "
                         f"{tuple(up.shape)}")
    _check_gated(x.shape[-1], block, bits_x, bits_w, act, compute_dtype)
    trust_x = default_trust(bits_x) if trust_x is None else trust_x
    trust_w = default_trust(bits_w) if trust_w is None else trust_w
    flat = _dense(x.reshape(-1, x.shape[-1]))
    gate, up = _dense(gate), _dense(up)
    h = QuestGatedFunction.apply(flat, gate, up, block, bits_x, bits_w, compute_dtype, act, trust_x, trust_w,
                                 _differentiates(flat, gate, up))
    return h.reshape(*x.shape[:-1], gate.shape[0])


class QuestFeedForward(torch.nn.Module):
    """Gated feed-forward block trained with QuEST quantisation: layer norm (optional; with mean and bias), the
    gated product of `width` columns, and a QuestLinear back to `features`.

    norm_act8: the norm keeps its normalised input in 8 bits for the backward
    pass.  ``freeze()`` quantises the three weights once and switches to eval
    mode, whose forwards then quantise activations only and carry no gradient;
    training mode, loading a state and moving the module drop the frozen operands.
    """

    def __init__(self, features: int, width: int, block: int = 128, bits_x: int = 4, bits_w: int = 4,
                 compute_dtype=torch.bfloat16, act: str = "silu", norm: bool = True, norm_act8: bool = True,
                 eps: float = 1e-5, trust_x: float | None = None, trust_w: float | None = None, device=None,
                 dtype=None):
        super().__init__()
        _check_gated(features, block, bits_x, bits_w, act, compute_dtype)
        self.block, self.bits_x, self.bits_w, self.act, self.compute_dtype = block, bits_x, bits_w, act, compute_dtype
        self.trust_x = default_trust(bits_x) if trust_x is None else trust_x
        self.trust_w = default_trust(bits_w) if trust_w is None else trust_w
        self.norm = LayerNorm(features, eps, act8=norm_act8, device=device, dtype=dtype) if norm else None
        self.gate = torch.nn.Parameter(torch.empty(width, features, device=device, dtype=dtype))
        self.up = torch.nn.Parameter(torch.empty(width, features, device=device, dtype=dtype))
        for w in (self.gate, self.up):
            torch.nn.init.kaiming_uniform_(w, a=5 ** 0.5)
        self.down = QuestLinear(width, features, bias=False, block=block, bits_x=bits_x, bits_w=bits_w,
                                compute_dtype=compute_dtype, trust_x=trust_x, trust_w=trust_w, device=device,
                                dtype=dtype)
        self._frozen = None

    def freeze(self) -> "QuestFeedForward":
        """Quantise the weights once and switch to eval mode; needs width a multiple of 128 as well."""
        self.down.freeze()
        with torch.no_grad():
            self._frozen = [(op, scale) for _, scale, _, op in
                            (quantize_fwd_op(_dense(w.detach()), self.block, self.bits_w, trust=self.trust_w)
                             for w in (self.gate, self.up))]
        return self.eval()

    def _thaw(self) -> None:
        self._frozen = None
        self.down._w_operand = self.down._w_scale = None

    def train(self, mode: bool = True) -> "QuestFeedForward":
        if mode:
            self._thaw()
        return super().train(mode)

    def _apply(self, *args, **kwargs):
        self._thaw()
        return super()._apply(*args, **kwargs)

    def _load_from_state_dict(self, *args, **kwargs):
        self._thaw()
        return super()._load_from_state_dict(*args, **kwargs)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if self.training or self._frozen is None:
            y = x if self.norm is None else self.norm(x)
            h = quest_gated(y, self.gate, self.up, self.block, self.bits_x, self.bits_w, self.compute_dtype, self.act,
                            self.trust_x, self.trust_w)
            return self.down(h)
        if x.shape[-1] != self.gate.shape[1]:
            raise ValueError(f"the last axis of x has {x.shape[-1]} entries, the block {self.gate.shape[1]}")
        with torch.no_grad():  # (the norm too: with a gradient to follow it would keep its checkpoint)
            y = x if self.norm is None else self.norm(x)
            flat = _dense(y.reshape(-1, y.shape[-1]))
            (go, gs), (uo, us) = self._frozen
            _, xs, _, xo = quantize_fwd_op(flat, self.block, self.bits_x, trust=self.trust_x)
            h, _, _ = gated_fwd(xo, xs, flat.shape[0], self.bits_x, go, gs, uo, us, self.gate.shape[0], self.bits_w,
                                flat.shape[1], act=self.act, out_dtype=self.compute_dtype)
        return self.down(h.reshape(*y.shape[:-1], h.shape[1]))
