"""A mixture of gated feed-forward experts around the products in 8-bit integers.

    out_t = sum over the top_k experts e of token t of p_te Q(h_te) Q(down_e)^T,
    h_te = act(Q(x_t) Q(gate_e)^T) * (Q(x_t) Q(up_e)^T)

with the quantiser of QuestLinear on every operand (the pages quantise the
inputs and weights of every linear layer: pith.science review of QuEST, "What
carries the argument").  Training runs each expert's products on its tokens
with quest_linear(int8=True).  Frozen, the layer of up to 64 tokens is one call
(quest_moe_fwd): routing, both products, the quantisation between them and the
sum over the experts, with the weights at 4 bits two in a byte.
"""
from __future__ import annotations

import math

import torch

from . import ACTIVATIONS, MOE_MAX_TOKENS, moe_fwd, quantize_fwd, quantize_fwd_i8
from .linear import _check_int8, _dense, default_trust, quest_linear

__all__ = ["QuestMoE", "route"]


def route(logits: torch.Tensor, top_k: int, over_all: bool = False):
    """(weights, experts) of each token, both (n, top_k), differentiable in the weights.

    The top_k largest logits, of equal ones the lowest index; weights are the
    softmax over them, or with over_all over all logits.  An expert with a
    logit of -infinity has the weight 0, also where the token has no other; a
    NaN or +infinity makes the token's weights NaN.
    """
    value, index = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
    none = value[:, :1] == -math.inf  # the largest
    value = value.masked_fill(none, 0.0)
    weight = torch.softmax(value if over_all else value[:, :top_k], dim=-1)[:, :top_k]
    return weight.masked_fill(none, 0.0), index[:, :top_k]


class QuestMoE(torch.nn.Module):
    """Gated experts of `width` columns with a router, trained with QuEST quantisation.

    Parameters: router (experts, features), gate_up (experts, 2 width,
    features), gate's rows first, and down (experts, features, width).  bits_h:
    of the products' input of down (bits_x by default).  ``freeze()`` quantises
    the weights once and switches to eval mode, whose forwards then quantise
    activations only and carry no gradient; more than 64 tokens are taken 64 at a
    time.  Training mode, loading a state and moving the module drop the frozen
    codes.  Frozen, what down multiplies is quantised from fp32, in training from
    compute_dtype.
    """

    def __init__(self, features: int, width: int, experts: int, top_k: int, block: int = 128, bits_x: int = 4,
                 bits_w: int = 4, bits_h: int | None = None, compute_dtype=torch.bfloat16, act: str = "silu",
                 over_all: bool = False, device=None, dtype=None):
        super().__init__()
        bits_h = bits_x if bits_h is None else bits_h
        for cols in (features, width):
            _check_int8("int", cols, bits_x, bits_w)
            if cols % block:
                raise ValueError(f"features and width ({features}, {width}) must be multiples of the Hadamard block "
                                 f"({block})")
        if not 1 <= bits_h <= 8:
            raise ValueError(f"bits_h is 1 to 8, not {bits_h}")
        if width > 8192 or not 1 <= experts <= 256 or not 1 <= top_k <= min(experts, 32):
            raise ValueError("width is at most 8192, experts 1 to 256 and top_k 1 to 32, at most experts: got "
                             f"{width}, {experts} and {top_k}")
        if act not in ACTIVATIONS:
            raise ValueError(f"act must be one of {tuple(ACTIVATIONS)}, not {act!r}")
        if compute_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"compute_dtype is float32 or bfloat16, not {compute_dtype}")
        self.block, self.bits_x, self.bits_w, self.bits_h = block, bits_x, bits_w, bits_h
        self.top_k, self.act, self.over_all, self.compute_dtype = top_k, act, over_all, compute_dtype
        self.router = torch.nn.Parameter(torch.empty(experts, features, device=device, dtype=dtype))
        self.gate_up = torch.nn.Parameter(torch.empty(experts, 2 * width, features, device=device, dtype=dtype))
        self.down = torch.nn.Parameter(torch.empty(experts, features, width, device=device, dtype=dtype))
        for w in (self.router, *self.gate_up.unbind(0), *self.down.unbind(0)):
            torch.nn.init.kaiming_uniform_(w.data, a=5 ** 0.5)
        self._frozen = None

    def _codes(self, w: torch.Tensor):
        """(codes, scales) of an (experts, rows, cols) weight, packed at 4 bits."""
        flat = _dense(w.detach().reshape(-1, w.shape[-1]))
        c, s = (quantize_fwd if self.bits_w == 4 else quantize_fwd_i8)(flat, self.block, self.bits_w)[:2]
        return c.reshape(*w.shape[:-1], -1), s.reshape(w.shape[:-1])

    def freeze(self) -> "QuestMoE":
        """Quantise the weights once and switch to eval mode."""
        width = self.down.shape[2]
        with torch.no_grad():
            codes, scale = self._codes(self.gate_up)
            self._frozen = (codes[:, :width].contiguous(), scale[:, :width].contiguous(),
                            codes[:, width:].contiguous(), scale[:, width:].contiguous(), *self._codes(self.down))
        return self.eval()

    def train(self, mode: bool = True) -> "QuestMoE":
        if mode:
            self._frozen = None
        return super().train(mode)

    def _apply(self, *args, **kwargs):
        self._frozen = None
        return super()._apply(*args, **kwargs)

    def _load_from_state_dict(self, *args, **kwargs):
        self._frozen = None
        return super()._load_from_state_dict(*args, **kwargs)

    def _linear(self, x, w, bits_x):
        return quest_linear(x, w, block=self.block, bits_x=bits_x, bits_w=self.bits_w,
                            compute_dtype=self.compute_dtype, trust_x=default_trust(bits_x),
                            trust_w=default_trust(self.bits_w), int8=True)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.router.shape[1]:
            raise ValueError(f"the last axis of x has {x.shape[-1]} entries, the layer {self.router.shape[1]}")
        flat = x.reshape(-1, x.shape[-1])
        if not self.training and self._frozen is not None:
            with torch.no_grad():
                parts = [self._few(_dense(t)) for t in flat.split(MOE_MAX_TOKENS)]
            return (parts[0] if len(parts) == 1 else torch.cat(parts)).reshape(x.shape)
        logits = torch.nn.functional.linear(flat.float(), self.router.float())
        weight, index = route(logits, self.top_k, self.over_all)
        index = index.masked_fill(logits.gather(-1, index) == -math.inf, -1)  # not taken
        # (a token's rows: in the order of its experts' index, whatever their rank)
        out = torch.zeros(flat.shape, dtype=torch.float32, device=x.device)
        taken = False
        # (unbound once: the backward pass of an expert's own select would write zeros for all of the others)
        for e, (gate_up, down) in enumerate(zip(self.gate_up.unbind(0), self.down.unbind(0))):
            token, rank = torch.nonzero(index == e, as_tuple=True)
            if not token.numel():
                continue
            taken = True
            g, u = self._linear(flat[token], gate_up, self.bits_x).float().chunk(2, -1)
            h = (torch.nn.functional.silu(g) if self.act == "silu" else torch.nn.functional.gelu(g)) * u
            y = self._linear(h.to(self.compute_dtype), down, self.bits_h)
            out = out.index_add(0, token, y.float() * weight[token, rank][:, None])
        if not taken:  # zeros, and so are the weights: a backward pass can follow all the same
            out = out + weight.sum()
        return out.to(self.compute_dtype).reshape(x.shape)

    def _few(self, x: torch.Tensor) -> torch.Tensor:
        logits = torch.nn.functional.linear(x.float(), self.router.float())
        codes, scale, _ = quantize_fwd_i8(x, self.block, self.bits_x)
        return moe_fwd(codes, scale, self.bits_x, logits, *self._frozen, self.bits_w, self.top_k, block=self.block,
                       h_bits=self.bits_h, act=self.act, over_all=self.over_all, out_dtype=self.compute_dtype)
