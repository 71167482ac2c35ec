"""Codes one a byte and their product in 8-bit integers, against the definitions in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantization_aware_amd as qa
from oracle import quest_oracle as qo
from parity import check_fwd
from quest_inputs import TensorSpec, make_tensor, to_float64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of fp32, relative


def log(msg: str) -> None:
    print(f"[gpu-i8] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    return torch.device("cuda", 0)


def rows_of(dev, rows, cols, dtype, seed):
    spec = TensorSpec("i8.x", rows, cols, dtype, "student_t", 4, seed, outlier_cols=max(1, cols // 100), outlier_scale=20.0)
    return make_tensor(spec, dev)


# ---------------------------------------------------------------------------
# The quantiser and its way back
# ---------------------------------------------------------------------------

QUANTISER = [(1, 64, 64, "bf16", 8), (3, 64, 64, "f32", 1), (513, 128, 128, "bf16", 5), (7, 192, 64, "f32", 6),
             (130, 256, 256, "bf16", 8), (300, 2048, 128, "bf16", 8), (33, 5632, 256, "f32", 8),
             (9, 5632, 128, "bf16", 7), (21, 960, 64, "bf16", 4), (5, 8192, 128, "bf16", 8), (2, 32768, 256, "f32", 8),
             (3, 32704, 64, "bf16", 2), (1030, 512, 128, "bf16", 3)]


@pytest.mark.parametrize("rows,cols,block,dtype,b", QUANTISER)
def test_quantiser(dev, rows, cols, block, dtype, b):
    log(f"quantise {rows}x{cols} block {block} {dtype} b={b}")
    x = rows_of(dev, rows, cols, dtype, rows + cols)
    trust = 1.3 if b == 1 else 1.0
    codes, scale, mask = qa.quantize_fwd_i8(x, block, b, trust=trust, with_mask=True)
    assert codes.dtype == torch.int8 and codes.shape == x.shape
    c = codes.cpu().numpy().astype(np.int64)
    half = 2 ** (b - 1)
    assert c.min() >= -half and c.max() < half
    packed = qo.pack_lsb_first((c + half).astype(np.uint8), b)
    stats = check_fwd(to_float64(x), block, b, packed, scale.cpu().numpy(), mask.cpu().numpy(), trust=trust)
    log(f"{stats['mismatched']} of {stats['elements']} differ")
    # without the mask, and into the caller's buffers: the same
    c2, s2, m2 = qa.quantize_fwd_i8(x, block, b, trust=trust, codes=torch.empty_like(codes))
    assert m2 is None and torch.equal(codes, c2) and torch.equal(scale, s2)
    # the values: the definition's, rounded (s / (2^b - 1), its product and the type's rounding)
    for out_dtype, extra in ((torch.float32, 0.0), (torch.bfloat16, torch.finfo(torch.bfloat16).eps / 2)):
        v = qa.dequantize_i8(codes, scale, b, out_dtype=out_dtype)
        want = (2 * c + 1) * scale.double().cpu().numpy()[:, None] / (2 ** b - 1)
        assert (np.abs(v.double().cpu().numpy() - want) <= np.abs(want) * (2.01 * U + extra * 1.01)).all()


def test_quantiser_zero_rows_and_rows_behind(dev):
    x = torch.zeros(40, 320, device=dev)
    x[1::2] = torch.randn(20, 320, device=dev)
    codes = torch.full((48, 320), 77, dtype=torch.int8, device=dev)
    scale = torch.full((48,), 7.0, device=dev)
    qa.quantize_fwd_i8(x, 64, 8, codes=codes[:40], scale=scale[:40])
    assert (codes[40:] == 77).all() and (scale[40:] == 7.0).all()
    assert (codes[:40:2] == 0).all() and (scale[:40:2] == 0).all()
    assert (qa.dequantize_i8(codes[:40], scale[:40], 8)[::2] == 0).all()
    assert torch.equal(codes[1], qa.quantize_fwd_i8(x[1:2].clone(), 64, 8)[0][0])


# ---------------------------------------------------------------------------
# The product
# ---------------------------------------------------------------------------

def coded(dev, rows, k, bits, seed, extreme=False):
    """(codes, scales): normal rows' codes, or the two ends of the range at random."""
    g = torch.Generator().manual_seed(seed)
    half = 2 ** (bits - 1)
    if extreme:
        c = torch.where(torch.rand((rows, k), generator=g) < 0.9, -half, half - 1)
    else:
        c = torch.floor(torch.randn((rows, k), generator=g) * half / 2.5).clamp(-half, half - 1)
    s = torch.exp(torch.randn((rows,), generator=g))
    return c.to(torch.int8).to(dev), s.to(dev)


def exact_product(a, sa, ab, b, sb, bb):
    """The product in 64 bits; the sums are whole numbers far below 2^53."""
    t = torch.matmul(2 * a.double() + 1, (2 * b.double() + 1).t())
    return t * (sa.double() / (2 ** ab - 1))[:, None] * (sb.double() / (2 ** bb - 1))


def check_product(y, want):
    """Roundings: 2 / (2^b - 1) and the step of both, the steps' product, the sum to fp32, the product; the type's."""
    out = torch.finfo(y.dtype).eps / 2 if y.dtype != torch.float32 else 0.0
    err = (y.double() - want).abs()
    bound = want.abs() * (7.01 * U + out * (1 + 8 * U))
    assert (err <= bound).all(), f"{float((err / bound.clamp(min=1e-300)).max()):.3g} of the bound"
    return float((err / bound.clamp(min=1e-300)).max())


SHAPES = [(1, 64, 1, 8, 8), (1, 2048, 2048, 8, 8), (2, 128, 17, 8, 5), (5, 192, 33, 7, 8), (16, 64, 8, 8, 8),
          (17, 1024, 40, 8, 8), (33, 448, 1001, 6, 8), (48, 2048, 512, 8, 8), (64, 960, 96, 8, 4), (65, 512, 260, 8, 8),
          (100, 896, 144, 3, 8), (128, 256, 1000, 8, 8), (129, 1152, 72, 8, 8), (255, 128, 130, 5, 7),
          (333, 960, 1001, 7, 5), (513, 704, 400, 8, 8), (1030, 64, 3, 8, 8), (2050, 320, 1, 8, 8), (3001, 192, 41, 8, 2),
          (1030, 256, 264, 8, 1), (2050, 384, 2112, 8, 8), (2049, 128, 2101, 8, 8), (130, 4224, 200, 8, 8),
          (70, 8192, 333, 8, 8), (4100, 576, 1288, 8, 8), (9, 32768, 64, 8, 8), (300, 32704, 70, 8, 8)]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k,n,ab,bb", SHAPES)
def test_product(dev, m, k, n, ab, bb, out_dtype):
    log(f"product {m}x{k}x{n} b={ab},{bb} {out_dtype}")
    (a, sa), (b, sb) = coded(dev, m, k, ab, m + k), coded(dev, n, k, bb, n + k + 1)
    y = qa.gemm_i8(a, sa, ab, b, sb, bb, out_dtype=out_dtype)
    assert y.shape == (m, n) and y.dtype == out_dtype
    log(f"error / tolerance {check_product(y, exact_product(a, sa, ab, b, sb, bb)):.3g}")


@pytest.mark.parametrize("m,k,n", [(3, 32768, 20), (200, 32768, 150), (1, 32704, 257)])
def test_sums_at_the_ends_of_their_range(dev, m, k, n):
    """Codes at the ends of 8 bits: sums up to 32768 255^2, terms of which pass 2^31."""
    log(f"ends {m}x{k}x{n}")
    (a, sa), (b, sb) = coded(dev, m, k, 8, 3, True), coded(dev, n, k, 8, 4, True)
    a[0], b[0] = -128, -128
    a[-1], b[-1] = 127, 127
    check_product(qa.gemm_i8(a, sa, 8, b, sb, 8, out_dtype=torch.float32), exact_product(a, sa, 8, b, sb, 8))


@pytest.mark.parametrize("m,n,k", [(5, 200, 256), (300, 264, 640)])
def test_equals_the_four_bit_product(dev, m, n, k):
    """Operands of 4 bits: the bits of quest_gemm's product of the same codes (sums below 2^24)."""
    xs = [torch.randn(r, k, device=dev).to(torch.bfloat16) for r in (m, n)]
    ops = [qa.quantize_fwd_op(x, 128, 4, with_codes=True) for x in xs]
    want = qa.gemm(ops[0][3], ops[0][1], m, 4, ops[1][3], ops[1][1], n, 4, k, out_dtype=torch.float32)
    bytes_ = []
    for codes, _, _, _ in ops:
        u = torch.stack([codes & 15, codes >> 4], -1).flatten(1).to(torch.int8) - 8
        bytes_.append(u.contiguous())
    got = qa.gemm_i8(bytes_[0], ops[0][1], 4, bytes_[1], ops[1][1], 4, out_dtype=torch.float32)
    assert torch.equal(got, want)


@pytest.mark.parametrize("m,n", [(1, 40), (40, 200), (300, 200), (300, 5), (700, 712)])
def test_rows_behind_the_last_are_left(dev, m, n):
    k = 192
    log(f"guard rows {m}x{n}")
    (a, sa), (b, sb) = coded(dev, m, k, 8, 5), coded(dev, n, k, 8, 6)
    buf = torch.full((m + 256, n), 7.0, dtype=torch.bfloat16, device=dev)
    y = qa.gemm_i8(a, sa, 8, b, sb, 8, out=buf[:m])
    assert (buf[m:] == 7.0).all()
    assert torch.equal(y, qa.gemm_i8(a, sa, 8, b, sb, 8))


def test_operand_with_itself_and_special_scales(dev):
    a, sa = coded(dev, 70, 256, 8, 7)
    y = qa.gemm_i8(a, sa, 8, a, sa, 8, out_dtype=torch.float32)
    assert torch.equal(y, y.t())
    sb = sa.clone()
    sb[3], sb[4], sb[5] = 0.0, float("inf"), float("nan")
    y = qa.gemm_i8(a, sa, 8, a, sb, 8, out_dtype=torch.float32)
    assert (y[:, 3] == 0).all() and y[:, 5].isnan().all() and not y[:, 4].isfinite().any()
    keep = [j for j in range(70) if j not in (3, 4, 5)]
    assert y[:, keep].isfinite().all()


def test_past_32_bit_offsets(dev):
    """Outputs and operands whose element offsets pass 2^31 and 2^32."""
    m, k, n = 131072 + 40, 32768, 24
    log("an operand of 2^32 bytes")
    a = torch.zeros((m, k), dtype=torch.int8, device=dev)
    a[-40:], sa = coded(dev, 40, k, 8, 8)[0], torch.ones(m, device=dev)
    b, sb = coded(dev, n, k, 8, 9)
    y = qa.gemm_i8(a, sa, 8, b, sb, 8, out_dtype=torch.float32)
    check_product(y[-40:], exact_product(a[-40:], sa[-40:], 8, b, sb, 8))
    y2 = qa.gemm_i8(b, sb, 8, a, sa, 8, out_dtype=torch.float32)
    assert torch.equal(y2, y.t())
    v = qa.dequantize_i8(a, sa, 8)
    assert torch.equal(v[-40:], qa.dequantize_i8(a[-40:], sa[-40:], 8))
    del a, v, y, y2
    m, n = 70000, 65000
    log("an output of 4.5 10^9 elements")
    (a, sa), (b, sb) = coded(dev, m, 64, 8, 10), coded(dev, n, 64, 8, 11)
    y = qa.gemm_i8(a, sa, 8, b, sb, 8)
    check_product(y[-300:, -300:], exact_product(a[-300:], sa[-300:], 8, b[-300:], sb[-300:], 8))
    check_product(y[33000:33100], exact_product(a[33000:33100], sa[33000:33100], 8, b, sb, 8))


@pytest.mark.parametrize("rows,cols,block", [(1, 64, 64), (3, 256, 256), (37, 320, 64), (1000, 1152, 128), (5, 32768, 256)])
def test_narrow_trust_backward(dev, rows, cols, block):
    """fp32 gradients to bf16: H (M G) of the formula in 64 bits, and the fp32 form's values rounded once."""
    log(f"narrow trust backward {rows}x{cols} block {block}")
    g = torch.Generator().manual_seed(rows + cols)
    grad = torch.randn(rows, cols, generator=g)
    grad[0, :block] *= 1e30
    mask = torch.randint(0, 256, (rows * cols // 8,), generator=g, dtype=torch.uint8)
    buf = torch.full((rows + 2, cols), 7.0, dtype=torch.bfloat16, device=dev)
    got = qa.trust_bwd_narrow(grad.to(dev), mask.to(dev), block, out=buf[:rows])
    assert (buf[rows:] == 7.0).all()
    assert torch.equal(got, qa.trust_bwd(grad.to(dev), mask.to(dev), block).to(torch.bfloat16))
    keep = np.unpackbits(mask.numpy(), bitorder="little").reshape(rows, cols)
    kept = (grad.double().numpy() * keep).reshape(rows, cols // block, block)
    had = np.array([[1.0]])
    while len(had) < block:
        had = np.block([[had, had], [had, -had]])
    want = (kept @ had / np.sqrt(block)).reshape(rows, cols)
    # log2(block) additions and the factor, each half a step of fp32 of at most the sum of magnitudes; then bf16's
    size = np.abs(kept).sum(-1, keepdims=True) / np.sqrt(block) * np.ones(block)
    bound = 2.0 ** -8 * np.abs(want) + 12 * U * size.reshape(rows, cols) * (1 + 2.0 ** -8)
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
    assert torch.equal(got, qa.trust_bwd_narrow(grad.to(dev), mask.to(dev), block))
    assert qa.trust_bwd_narrow(grad[:0].to(dev), mask[:0].to(dev), block).shape == (0, cols)
