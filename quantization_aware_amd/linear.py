"""QuEST quantisation-aware linear layer on libquest.

y = Q(x) Q(w)^T + bias, where Q(.) quantises each operand along the
contraction axis (blockwise Hadamard transform, RMS clip scale, b-bit grid)
and returns the grid values in the Hadamard domain.  The transform is
orthogonal and applied to both operands, so the product of the transformed
operands equals the product of their original-domain reconstructions
(pith.science review of QuEST, "Assumptions & free parameters").  The
backward pass uses the trust estimator on both operands: the gradient
reaching Q(x) is dy Q(w), the one reaching Q(w) is dy^T Q(x); each is masked
by its operand's trust mask and transformed back (pith.science review,
"What carries the argument" and the Figure 2 caption).

Quantisation, masking and both transforms run in libquest's kernels
(quest_quantize_fwd_ex, or the FP4 and 2:4-sparse forwards, and
quest_trust_bwd).  On the int grid with b <= 4 and K a multiple of 128 the
forward product is libquest's FP6 product of the two operands
(quest_quantize_fwd_op with codes and mask, both operands in one
quest_quantize_fwd_op_group launch when they share dtype and trust factor,
then quest_gemm: exact sums, one rounding to the compute dtype), and the backward rebuilds Q(x) and Q(w) from
the saved codes (quest_dequantize, the same values as the dequantised
forward output).  The two gradient products, and the forward product of the
other configurations, are plain library GEMMs through torch.  ``grid`` picks the format the operands are quantised to: "int"
(b-bit midrise levels), "fp4" (E2M1 levels, 4 bits whatever bits_x and
bits_w say) or "sparse24" (2:4-sparse b-bit levels), the formats the pages
train with (pith.science review of QuEST, the list of contributions and the
captions of Figures 3 and 4); all three share the transform, the RMS scale
and the trust rule.

Inference (``QuestLinear.freeze``, then eval mode): the weight is quantised
once into the FP6 matrix-core operand, each activation by
quest_quantize_fwd_op, and the product is libquest's FP6 GEMM (quest_gemm):
the 4-bit layer product whose speed the pages compare with BF16 (pith.science
review, Figure 5 caption).

``int8``: products in 8-bit integers, for 1 to 8 bits on the "int" grid (the
pages train W8A8 models as well: pith.science review of QuEST, Figure 8
caption).  Both operands are quantised to codes one a byte (quest_quantize_fwd_i8)
and the forward product is quest_gemm_i8, with exact sums and one rounding to
the compute dtype, where the default above 4 bits rounds both operands' values
to the compute dtype first.  The backward rebuilds them (quest_dequantize_i8) for
the same two gradient products, whose fp32 sums are rounded once, behind the trust
backward (quest_trust_bwd_narrow).  ``freeze`` then keeps the weight's codes.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (dequantize, dequantize_i8, gemm, gemm_i8, quantize_fwd_ex, quantize_fwd_fp4, quantize_fwd_i8,
               quantize_fwd_op, quantize_fwd_op_group, quantize_fwd_sparse24, trust_bwd, trust_bwd_narrow)

__all__ = ["QuestLinearFunction", "QuestLinearInt8Function", "quest_linear", "quest_linear_operand",
           "quest_linear_int8", "QuestLinear", "default_trust", "ONE_BIT_OUTER_TRUST", "GRIDS"]


ONE_BIT_OUTER_TRUST = 1.30  # pith.science review of QuEST, "Assumptions & free parameters" (s*)
GRIDS = ("int", "fp4", "sparse24")


def _check_grid(grid: str) -> None:
    if grid not in GRIDS:
        raise ValueError(f"grid must be one of {GRIDS}, not {grid!r}")


def _quantise(t: torch.Tensor, block: int, bits: int, trust: float, grid: str, dtype):
    """(trust mask, dequantised Hadamard-domain values in dtype) of t on the chosen grid."""
    if grid == "int":
        _, _, mask, q = quantize_fwd_ex(t, block, bits, trust=trust, with_codes=False, dq_dtype=dtype)
    elif grid == "fp4":
        _, _, mask, q = quantize_fwd_fp4(t, block, trust, with_codes=False, dq_dtype=dtype)
    else:
        _, _, _, mask, q = quantize_fwd_sparse24(t, block, bits, trust, with_codes=False, dq_dtype=dtype)
    return mask, q


def default_trust(bits: int) -> float:
    """Outer trust factor used when none is given: 1.30 at 1 bit, 1 otherwise."""
    return ONE_BIT_OUTER_TRUST if bits == 1 else 1.0


class QuestLinearFunction(torch.autograd.Function):
    """y = Q(x) Q(w)^T for 2-D x (N x K) and w (M x K), K a multiple of `block`."""

    @staticmethod
    def forward(ctx, x, w, block, bits_x, bits_w, compute_dtype, trust_x=1.0, trust_w=1.0, grid="int"):
        ctx.block = block
        ctx.x_dtype, ctx.w_dtype = x.dtype, w.dtype
        # the FP6 product's domain: midrise levels of at most 4 bits, k a multiple of 128 up to 65536
        # (exact fp32 sums), at most 2^20 output features
        ctx.fp6 = (grid == "int" and max(bits_x, bits_w) <= 4 and x.shape[1] % 128 == 0 and x.shape[1] <= 65536
                   and 0 < w.shape[0] <= 2 ** 20 and 0 < x.shape[0] <= 2 ** 30)
        if ctx.fp6:
            n, k = x.shape
            m = w.shape[0]
            # With one bit width and n a multiple of 4 (every buffer 16-byte
            # aligned), the codes, scales and masks of x and w are the rows of
            # one (n + m)-row tensor each, so that the backward rebuilds both
            # operands in one quest_dequantize launch.
            ctx.joint = bits_x == bits_w and n % 4 == 0
            if ctx.joint:
                dev = x.device
                codes = torch.empty((n + m, k * bits_x // 8), dtype=torch.uint8, device=dev)
                scale = torch.empty((n + m,), dtype=torch.float32, device=dev)
                mask = torch.empty((n + m, k // 8), dtype=torch.uint8, device=dev)
                outs = [dict(codes=codes[:n], scale=scale[:n], mask=mask[:n]),
                        dict(codes=codes[n:], scale=scale[n:], mask=mask[n:])]
                if trust_x == trust_w and x.dtype == w.dtype:
                    # one launch for both operands (quest_quantize_fwd_op_group)
                    (cx, sx, mask_x, ox), (cw, sw, mask_w, ow) = quantize_fwd_op_group([x, w], block, bits_x,
                                                                                      trust=trust_x, outs=outs)
                else:
                    cx, sx, mask_x, ox = quantize_fwd_op(x, block, bits_x, trust=trust_x, **outs[0])
                    cw, sw, mask_w, ow = quantize_fwd_op(w, block, bits_w, trust=trust_w, **outs[1])
            else:
                cx, sx, mask_x, ox = quantize_fwd_op(x, block, bits_x, trust=trust_x, with_codes=True,
                                                     with_mask=True)
                cw, sw, mask_w, ow = quantize_fwd_op(w, block, bits_w, trust=trust_w, with_codes=True,
                                                     with_mask=True)
            out_dtype = torch.float32 if compute_dtype == torch.float32 else torch.bfloat16
            y = gemm(ox, sx, n, bits_x, ow, sw, m, bits_w, k, out_dtype=out_dtype)
            y = y.to(compute_dtype)
            if ctx.joint:
                ctx.save_for_backward(codes, scale, mask)
            else:
                ctx.save_for_backward(cx, sx, cw, sw, mask_x, mask_w)
            ctx.dims = (n, m, k, bits_x, bits_w, compute_dtype)
            return y
        mask_x, qx = _quantise(x, block, bits_x, trust_x, grid, compute_dtype)
        mask_w, qw = _quantise(w, block, bits_w, trust_w, grid, compute_dtype)
        y = torch.nn.functional.linear(qx, qw)
        ctx.save_for_backward(qx, qw, mask_x, mask_w)
        return y

    @staticmethod
    def backward(ctx, dy):
        if ctx.fp6 and ctx.joint and ctx.needs_input_grad[0] and ctx.needs_input_grad[1]:
            return QuestLinearFunction._backward_joint(ctx, dy)
        if ctx.fp6:
            if ctx.joint:
                codes, scale, mask = ctx.saved_tensors
                n = ctx.dims[0]
                cx, sx, mask_x, cw, sw, mask_w = codes[:n], scale[:n], mask[:n], codes[n:], scale[n:], mask[n:]
            else:
                cx, sx, cw, sw, mask_x, mask_w = ctx.saved_tensors
            n, m, k, bits_x, bits_w, compute_dtype = ctx.dims
            # Q(x) for the weight gradient and Q(w) for the input gradient,
            # rebuilt from the codes (both first: the rebuilds keep the GPU
            # busy while the host sets up the products)
            qx = dequantize(cx, sx, n, k, bits_x, out_dtype=compute_dtype) if ctx.needs_input_grad[1] else None
            qw = dequantize(cw, sw, m, k, bits_w, out_dtype=compute_dtype) if ctx.needs_input_grad[0] else None
        else:
            qx, qw, mask_x, mask_w = ctx.saved_tensors
            compute_dtype = qx.dtype
        dy = dy.to(compute_dtype).contiguous()
        dx = dw = None
        # The weight gradient first: its product reads Q(x) just after the
        # rebuild wrote it, while it is still in the last-level cache.
        if ctx.needs_input_grad[1]:
            # gradient reaching Q(w), Hadamard domain (a 2-D product with a
            # transposed left operand, as torch's own linear backward computes it)
            g = torch.mm(dy.t(), qx)
            dw = trust_bwd(g, mask_w, ctx.block, out=g).to(ctx.w_dtype)
        if ctx.needs_input_grad[0]:
            g = torch.mm(dy, qw)  # gradient reaching Q(x), Hadamard domain
            dx = trust_bwd(g, mask_x, ctx.block, out=g).to(ctx.x_dtype)
        return dx, dw, None, None, None, None, None, None, None

    @staticmethod
    def _backward_joint(ctx, dy):
        """Both gradients of the FP6 path, x's and w's state held as the rows of one tensor each.

        One rebuild launch gives [Q(x); Q(w)]; the weight gradient comes first,
        while Q(x) is still in the last-level cache.  Each gradient is masked
        and transformed back in a buffer of its own: the weight's outlives the
        step, and as rows of a joint one would keep the input's with it.
        """
        codes, scale, mask = ctx.saved_tensors
        n, m, k, bits, _, compute_dtype = ctx.dims
        q = dequantize(codes, scale, n + m, k, bits, out_dtype=compute_dtype)
        qx, qw = q[:n], q[n:]
        dy = dy.to(compute_dtype).contiguous()
        # gradients reaching Q(w) and Q(x), Hadamard domain (the weight's as a
        # 2-D product with a transposed left operand, as torch's own linear
        # backward computes it)
        gw = torch.mm(dy.t(), qx)
        gx = torch.mm(dy, qw)
        trust_bwd(gw, mask[n:], ctx.block, out=gw)
        trust_bwd(gx, mask[:n], ctx.block, out=gx)
        return gx.to(ctx.x_dtype), gw.to(ctx.w_dtype), None, None, None, None, None, None, None


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t contiguous and on a 16-byte boundary (a view into a tensor may be neither), as the library takes it."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _product_dtype(compute_dtype):
    """What a product writes: fp32 for fp32, bf16 for every other compute dtype (converted after it)."""
    return torch.float32 if compute_dtype == torch.float32 else torch.bfloat16


class QuestLinearInt8Function(torch.autograd.Function):
    """y = Q(x) Q(w)^T for 2-D x (N x K) and w (M x K) in 8-bit integers, K a multiple of `block`."""

    @staticmethod
    def forward(ctx, x, w, block, bits_x, bits_w, compute_dtype, trust_x, trust_w, keep):
        (n, k), m, dev = x.shape, w.shape[0], x.device
        # As in QuestLinearFunction: with one bit width and n a multiple of 4 the codes, scales and
        # masks of x and w are the rows of one tensor each, for one rebuild.
        ctx.joint = keep and bits_x == bits_w and n % 4 == 0
        outs = [{}, {}]
        if ctx.joint:
            codes = torch.empty((n + m, k), dtype=torch.int8, device=dev)
            scale = torch.empty((n + m,), dtype=torch.float32, device=dev)
            mask = torch.empty((n + m, k // 8), dtype=torch.uint8, device=dev)
            outs = [dict(codes=codes[:n], scale=scale[:n], mask=mask[:n]),
                    dict(codes=codes[n:], scale=scale[n:], mask=mask[n:])]
        cx, sx, mx = quantize_fwd_i8(x, block, bits_x, trust_x, with_mask=keep, **outs[0])
        cw, sw, mw = quantize_fwd_i8(w, block, bits_w, trust_w, with_mask=keep, **outs[1])
        if ctx.joint:
            ctx.save_for_backward(codes, scale, mask)
        elif keep:
            ctx.save_for_backward(cx, sx, mx, cw, sw, mw)
        ctx.dims = (n, m, k, block, bits_x, bits_w, compute_dtype)
        ctx.dtypes = (x.dtype, w.dtype)
        return gemm_i8(cx, sx, bits_x, cw, sw, bits_w, out_dtype=_product_dtype(compute_dtype)).to(compute_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        n, m, k, block, bits_x, bits_w, compute_dtype = ctx.dims
        need_x, need_w = ctx.needs_input_grad[:2]
        if ctx.joint:
            codes, scale, mask = ctx.saved_tensors
            cx, sx, mx, cw, sw, mw = codes[:n], scale[:n], mask[:n], codes[n:], scale[n:], mask[n:]
        else:
            cx, sx, mx, cw, sw, mw = ctx.saved_tensors
        dtype = _product_dtype(compute_dtype)
        dy = dy.to(dtype).contiguous()
        wide = {} if dtype == torch.float32 else {"out_dtype": torch.float32}

        def masked(g, mask, to):
            return trust_bwd_narrow(g, mask, block) if to == torch.bfloat16 else trust_bwd(g, mask, block, out=g)

        # The products' sums stay in fp32 up to the gradients' own type: rounded to bf16 both before and after the
        # transform, and Q before the product, the gradients were 0.0029 off instead of 0.0023 (a rounding is 0.0017).
        # Each gradient has a buffer of its own: the weight's is kept behind the step, and as rows of a joint one it
        # would keep the input's rows as well (151 MB for 16.8 MB at 16384 x 2048 -> 2048 in fp32).
        if ctx.joint and need_x and need_w:
            q = dequantize_i8(codes, scale, bits_x, out_dtype=dtype)
            qx, qw = q[:n], q[n:]
        else:
            qx = dequantize_i8(cx, sx, bits_x, out_dtype=dtype) if need_w else None
            qw = dequantize_i8(cw, sw, bits_w, out_dtype=dtype) if need_x else None
        # (the weight's first, as in QuestLinearFunction)
        dw = masked(torch.mm(dy.t(), qx, **wide), mw, ctx.dtypes[1]) if need_w else None
        dx = masked(torch.mm(dy, qw, **wide), mx, ctx.dtypes[0]) if need_x else None
        return dx, dw, *(None,) * 7


def _check_int8(grid: str, in_features: int, bits_x: int, bits_w: int) -> None:
    if grid != "int" or not (1 <= bits_x <= 8 and 1 <= bits_w <= 8) or in_features > 32768:
        raise ValueError("products in 8-bit integers need the int grid, 1 to 8 bits and at most 32768 in_features: got "
                         f"{grid!r}, {bits_x} and {bits_w} bits, {in_features} in_features")


def quest_linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None, block: int = 128,
                 bits_x: int = 4, bits_w: int = 4, compute_dtype=torch.bfloat16, trust_x: float | None = None,
                 trust_w: float | None = None, grid: str = "int", int8: bool = False) -> torch.Tensor:
    """QuEST linear map of x (..., K) by w (M, K); leading axes of x are flattened.

    trust_x / trust_w: outer trust factors; by default 1.30 for 1-bit operands
    of the "int" grid (the factor the pages tune for their 1-bit runs) and 1
    otherwise.  grid: "int", "fp4" or "sparse24".  int8: the product in 8-bit
    integers (1 to 8 bits, the "int" grid).
    """
    _check_grid(grid)
    trust_x = (default_trust(bits_x) if grid == "int" else 1.0) if trust_x is None else trust_x
    trust_w = (default_trust(bits_w) if grid == "int" else 1.0) if trust_w is None else trust_w
    lead = x.shape[:-1]
    if int8:
        _check_int8(grid, x.shape[-1], bits_x, bits_w)
        flat = x.dim() == 2  # (views both ways cost a small step some 15 us on the host)
        x2, w2 = _dense(x if flat else x.reshape(-1, x.shape[-1])), _dense(w)
        keep = torch.is_grad_enabled() and (x2.requires_grad or w2.requires_grad)
        y = QuestLinearInt8Function.apply(x2, w2, block, bits_x, bits_w, compute_dtype, trust_x, trust_w, keep)
        if bias is not None:
            y = y + bias.to(y.dtype)
        return y if flat else y.reshape(*lead, w.shape[0])
    x2 = x.reshape(-1, x.shape[-1]).contiguous()
    y = QuestLinearFunction.apply(x2, w.contiguous(), block, bits_x, bits_w, compute_dtype, trust_x, trust_w, grid)
    if bias is not None:
        y = y + bias.to(y.dtype)
    return y.reshape(*lead, w.shape[0])


def quest_linear_operand(x: torch.Tensor, w_operand: torch.Tensor, w_scale: torch.Tensor, out_features: int,
                         bits_w: int, bias: torch.Tensor | None = None, block: int = 128, bits_x: int = 4,
                         out_dtype=torch.bfloat16) -> torch.Tensor:
    """Inference product Q(x) Q(w)^T (+ bias) with w already in operand form.

    x (..., K) bf16 or fp32 with K a multiple of 128; w_operand / w_scale as
    returned by quantize_fwd_op for the (out_features x K) weight at bits_w.
    The activation is quantised (b = bits_x <= 4) straight into its operand
    and multiplied on the matrix cores; no gradient flows but the bias's.
    """
    lead = x.shape[:-1]
    k = x.shape[-1]
    x2 = x.reshape(-1, k).contiguous()
    _, x_scale, _, x_op = quantize_fwd_op(x2, block, bits_x)
    y = gemm(x_op, x_scale, x2.shape[0], bits_x, w_operand, w_scale, out_features, bits_w, k, out_dtype=out_dtype)
    if bias is not None:
        y = y + bias.to(y.dtype)
    return y.reshape(*lead, out_features)


def quest_linear_int8(x: torch.Tensor, w_codes: torch.Tensor, w_scale: torch.Tensor, bits_w: int,
                      bias: torch.Tensor | None = None, block: int = 128, bits_x: int = 8,
                      out_dtype=torch.bfloat16) -> torch.Tensor:
    """Inference product Q(x) Q(w)^T (+ bias) in 8-bit integers, with w already quantised.

    x (..., K) bf16 or fp32; w_codes (M, K) int8 and w_scale (M,) as returned
    by quantize_fwd_i8 at bits_w.  out_dtype: any floating-point type, as
    quest_linear's compute_dtype.  No gradient flows.
    """
    if not (isinstance(out_dtype, torch.dtype) and out_dtype.is_floating_point):
        raise TypeError(f"out_dtype must be a floating-point type, not {out_dtype}")
    x2 = _dense(x.detach().reshape(-1, x.shape[-1]))
    cx, sx, _ = quantize_fwd_i8(x2, block, bits_x)
    y = gemm_i8(cx, sx, bits_x, w_codes, w_scale, bits_w, out_dtype=_product_dtype(out_dtype)).to(out_dtype)
    if bias is not None:
        y = y + bias.detach().to(y.dtype)
    return y.reshape(*x.shape[:-1], w_codes.shape[0])


class QuestLinear(torch.nn.Module):
    """Drop-in linear layer trained with QuEST quantisation of weights and activations (int8: as in quest_linear)."""

    int8 = False  # (of modules pickled before there was the choice)

    def __init__(self, in_features: int, out_features: int, bias: bool = True, block: int = 128, bits_x: int = 4,
                 bits_w: int = 4, compute_dtype=torch.bfloat16, trust_x: float | None = None,
                 trust_w: float | None = None, grid: str = "int", device=None, dtype=None, int8: bool = False):
        super().__init__()
        if in_features % block:
            raise ValueError(f"in_features ({in_features}) must be a multiple of the Hadamard block ({block})")
        _check_grid(grid)
        if int8:
            _check_int8(grid, in_features, bits_x, bits_w)
        self.int8 = int8
        self.block, self.bits_x, self.bits_w, self.compute_dtype = block, bits_x, bits_w, compute_dtype
        self.grid = grid
        self.trust_x = (default_trust(bits_x) if grid == "int" else 1.0) if trust_x is None else trust_x
        self.trust_w = (default_trust(bits_w) if grid == "int" else 1.0) if trust_w is None else trust_w
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(out_features, device=device, dtype=dtype)) if bias else None
        torch.nn.init.kaiming_uniform_(self.weight, a=5 ** 0.5)
        self._w_operand = self._w_scale = None

    def freeze(self) -> "QuestLinear":
        """Quantise the weight once into the FP6 operand and switch to eval mode; eval-mode
        forwards then run the matrix-core product.  Needs bits_x, bits_w <= 4 and
        in_features a multiple of 128, on the "int" grid; training mode (``train()``) drops the operand.
        With int8 the weight's codes are kept instead, and the product is the one in 8-bit integers; loading a
        state and moving the module drop them as well."""
        if self.int8:
            with torch.no_grad():
                self._w_operand, self._w_scale, _ = quantize_fwd_i8(_dense(self.weight.detach()), self.block,
                                                                    self.bits_w)
            return self.eval()
        if self.grid != "int" or max(self.bits_x, self.bits_w) > 4 or self.weight.shape[1] % 128:
            raise ValueError("the FP6 product needs the int grid, bits <= 4 and in_features a multiple of 128")
        with torch.no_grad():
            _, self._w_scale, _, self._w_operand = quantize_fwd_op(self.weight.detach().contiguous(), self.block,
                                                                   self.bits_w)
        return self.eval()

    def train(self, mode: bool = True) -> "QuestLinear":
        if mode:
            self._w_operand = self._w_scale = None
        return super().train(mode)

    def _apply(self, *args, **kwargs):
        if self.int8:
            self._w_operand = self._w_scale = None
        return super()._apply(*args, **kwargs)

    def _load_from_state_dict(self, *args, **kwargs):
        if self.int8:
            self._w_operand = self._w_scale = None
        return super()._load_from_state_dict(*args, **kwargs)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if not self.training and self._w_operand is not None:
            if self.int8:
                return quest_linear_int8(x, self._w_operand, self._w_scale, self.bits_w, self.bias, self.block,
                                         self.bits_x, self.compute_dtype)
            return quest_linear_operand(x, self._w_operand, self._w_scale, self.weight.shape[0], self.bits_w,
                                        self.bias, self.block, self.bits_x, _product_dtype(self.compute_dtype))
        return quest_linear(x, self.weight, self.bias, self.block, self.bits_x, self.bits_w, self.compute_dtype,
                            self.trust_x, self.trust_w, self.grid, self.int8)
