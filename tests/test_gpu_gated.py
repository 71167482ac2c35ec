"""The gated product and its backward against the definition in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import feedforward_oracle as fo
import quantization_aware_amd as qa

pytestmark = pytest.mark.gpu


def log(msg: str) -> None:
    print(f"[gpu-gated] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    return torch.device("cuda", 0)


def quantised(dev, rows, k, bits, seed, std=1.0):
    """(operand, scale, exact levels) of a quantised normal tensor."""
    g = torch.Generator().manual_seed(seed)
    t = (std * torch.randn((rows, k), generator=g)).to(torch.bfloat16).to(dev)
    codes, scale, _, op = qa.quantize_fwd_op(t, 128, bits, with_codes=True)
    return op, scale, fo.Levels(fo.unpacked(codes, rows, k, bits), scale.cpu().numpy(), bits)


def case(dev, n, k, m, xb, wb, seed=1):
    return (quantised(dev, n, k, xb, seed), quantised(dev, m, k, wb, seed + 1, k ** -0.5),
            quantised(dev, m, k, wb, seed + 2, k ** -0.5))


def call(ops, n, k, m, xb, wb, **kw):
    (xo, xs, _), (go, gs, _), (uo, us, _) = ops
    return qa.gated_fwd(xo, xs, n, xb, go, gs, uo, us, m, wb, k, **kw)


SHAPES = [(1, 128, 1, 4, 4), (1, 2048, 5632, 4, 4), (3, 256, 40, 2, 3), (17, 128, 33, 1, 1), (32, 640, 1001, 3, 2),
          (33, 384, 128, 4, 4), (48, 2048, 512, 4, 4), (64, 1024, 96, 4, 2), (65, 512, 260, 4, 4), (100, 896, 144, 2, 4),
          (128, 256, 1000, 4, 4), (129, 1152, 72, 4, 4), (255, 128, 130, 3, 3), (300, 640, 1001, 3, 2),
          (513, 768, 400, 4, 4), (1030, 256, 264, 4, 1), (2050, 384, 2112, 4, 4), (2049, 128, 2101, 4, 3), (130, 4224, 200, 4, 4), (70, 4480, 333, 3, 4)]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("n,k,m,xb,wb", SHAPES)
def test_forward(dev, n, k, m, xb, wb, act, out_dtype):
    log(f"forward {n}x{k}x{m} b={xb},{wb} {act} {out_dtype}")
    ops = case(dev, n, k, m, xb, wb, seed=n + k + m)
    h, g8, u8 = call(ops, n, k, m, xb, wb, act=act, out_dtype=out_dtype)
    assert g8 is None and u8 is None
    want, g, u, err, dg, du = fo.gated_fwd(ops[0][2], ops[1][2], ops[2][2], act)
    r = fo.check("h", h, want, err)
    log(f"error / tolerance {r:.3g}")
    # the training form: the same h, and the checkpoints of the products that quest_gemm gives
    h2, g8, u8 = call(ops, n, k, m, xb, wb, act=act, out_dtype=out_dtype, act8=True)
    assert torch.equal(h, h2)
    for (codes, scale), exact, d, (wo, ws, _) in ((g8, g, dg, ops[1]), (u8, u, du, ops[2])):
        fo.check_act8_of(codes.cpu().numpy(), scale.cpu().numpy(), exact, d)
        prod = qa.gemm(ops[0][0], ops[0][1], n, xb, wo, ws, m, wb, k, out_dtype=torch.float32)
        c, s = qa.act8_save(prod)
        assert torch.equal(codes, c) and torch.equal(scale, s)


@pytest.mark.parametrize("n", [1, 40, 300])
def test_rows_behind_the_last_are_left(dev, n):
    """Only the n x m outputs are written, also where a tile reaches past them."""
    k, m = 256, 200
    log(f"guard rows, n={n}")
    ops = case(dev, n, k, m, 4, 4)
    buf = torch.full((n + 256, m), 7.0, dtype=torch.bfloat16, device=dev)
    h, _, _ = call(ops, n, k, m, 4, 4, out=buf[:n])
    assert (buf[n:] == 7.0).all()
    assert torch.equal(h, call(ops, n, k, m, 4, 4)[0])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_wide_values(dev, act):
    """Products far outside the activation's curved part, of both signs."""
    log(f"wide values, {act}")
    n, k, m = 40, 256, 64
    ops = (quantised(dev, n, k, 4, 1, 3.0), quantised(dev, m, k, 4, 2, 1.0), quantised(dev, m, k, 4, 3, 1.0))
    for dt in (torch.bfloat16, torch.float32):
        h, _, _ = call(ops, n, k, m, 4, 4, act=act, out_dtype=dt)
        want, _, _, err, _, _ = fo.gated_fwd(ops[0][2], ops[1][2], ops[2][2], act)
        # values that underflow fp32 on the way (act(g) below the smallest normal number) may be lost
        fo.check("h", h, want, err + 2.0 ** -126 * (1 + np.abs(ops[0][2].times(ops[2][2]))))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("n,k,m", [(40, 256, 200), (64, 128, 96), (65, 128, 96), (300, 256, 200), (300, 128, 208),
                                   (70, 4224, 150), (2309, 128, 2320), (2305, 128, 2317)])
def test_checkpoints_of_bad_products(dev, n, k, m, act):
    """Clip scales with infinities, NaN and values whose products overflow: the checkpoints are those that the products
    give when they are saved (a block with such an entry: exponent 255, codes 0), at every number of rows, and the
    backward pass gives NaN in those blocks and nowhere else."""
    log(f"bad products {n}x{k}x{m} {act}")
    (xo, xs, _), (go, gs, _), (uo, us, _) = case(dev, n, k, m, 4, 4, seed=n + m)
    xs, gs, us = xs.clone(), gs.clone(), us.clone()
    xs[3], xs[n - 1], xs[n // 2] = float("nan"), float("inf"), 1e30
    gs[5], gs[m - 1], us[40], us[m // 2] = float("nan"), 1e30, float("inf"), float("-inf")
    _, g8, u8 = qa.gated_fwd(xo, xs, n, 4, go, gs, uo, us, m, 4, k, act=act, act8=True)
    bad = []
    for (codes, scale), wo, ws in ((g8, go, gs), (u8, uo, us)):
        prod = qa.gemm(xo, xs, n, 4, wo, ws, m, 4, k, out_dtype=torch.float32)
        c, s = qa.act8_save(prod)
        assert torch.equal(scale, s) and torch.equal(codes, c)
        bad.append(s == 255)
        pad = torch.nn.functional.pad(~torch.isfinite(prod), (0, -m % 32)).reshape(n, -1, 32).any(2)
        assert torch.equal(bad[-1], pad) and pad.any() and not pad.all()
    wide = [b.repeat_interleave(32, dim=1)[:, :m] for b in bad]
    dh = torch.full((n, m), 1e-3, device=dev)
    out = qa.gated_bwd(dh, g8, u8, act=act)
    assert torch.equal(torch.isnan(out), torch.cat([wide[0] | wide[1], wide[0]], 1))


# (products of 128 x 128 tiles need five tiles for every four of the 256 compute units)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("n,k,m,xb,wb", [(2309, 256, 2320, 4, 4), (2305, 384, 2317, 3, 4), (40961, 128, 65, 4, 4)])
def test_forward_of_many_tiles(dev, n, k, m, xb, wb, act, out_dtype):
    """Products large enough for the largest tiles, of widths with and without whole 16-byte chunks."""
    log(f"many tiles {n}x{k}x{m} b={xb},{wb} {act} {out_dtype}")
    ops = case(dev, n, k, m, xb, wb, seed=n + k + m)
    h, _, _ = call(ops, n, k, m, xb, wb, act=act, out_dtype=out_dtype)
    g, u = ops[0][2].times(ops[1][2]), ops[0][2].times(ops[2][2])
    # fp32 roundings of a product: 2 / (2^b - 1) and its product with the clip scale for both operands, the product
    # of the two, and that with the exact sum
    dg, du = 6 * fo.U * np.abs(g), 6 * fo.U * np.abs(u)
    v, slope, dv, _ = fo.act(g, act)
    d_act = dv + np.abs(slope) * dg + dg * dg
    r = fo.check("h", h, v * u, np.abs(u) * d_act + (np.abs(v) + d_act) * du + 2 * fo.U * np.abs(v * u))
    log(f"error / tolerance {r:.3g}")
    h2, g8, u8 = call(ops, n, k, m, xb, wb, act=act, out_dtype=out_dtype, act8=True)
    assert torch.equal(h, h2)
    for (codes, scale), exact, d, (wo, ws, _) in ((g8, g, dg, ops[1]), (u8, u, du, ops[2])):
        fo.check_act8_of(codes.cpu().numpy(), scale.cpu().numpy(), exact, d)
        c, s = qa.act8_save(qa.gemm(ops[0][0], ops[0][1], n, xb, wo, ws, m, wb, k, out_dtype=torch.float32))
        assert torch.equal(codes, c) and torch.equal(scale, s)


def test_zero_rows_and_shared_weights(dev):
    log("zero rows, gate and up one buffer")
    n, k, m = 20, 256, 48
    x = torch.randn((n, k)).to(torch.bfloat16)
    x[5] = 0
    codes, xs, _, xo = qa.quantize_fwd_op(x.to(dev), 128, 4, with_codes=True)
    w = quantised(dev, m, k, 4, 5, k ** -0.5)
    h, g8, u8 = qa.gated_fwd(xo, xs, n, 4, w[0], w[1], w[0], w[1], m, 4, k, act8=True)
    assert not h[5].any() and torch.equal(g8[0], u8[0]) and not g8[0][5].any() and not g8[1][5].any()
    q = fo.Levels(fo.unpacked(codes, n, k, 4), xs.cpu().numpy(), 4)
    want, _, _, err, _, _ = fo.gated_fwd(q, w[2], w[2], "silu")
    fo.check("h", h, want, err)


def test_empty(dev):
    log("empty")
    e8, e32 = torch.empty(0, dtype=torch.uint8, device=dev), torch.empty(0, device=dev)
    w = quantised(dev, 40, 256, 4, 5)
    h, _, _ = qa.gated_fwd(e8, e32, 0, 4, w[0], w[1], w[0], w[1], 40, 4, 256)
    assert h.shape == (0, 40)
    h, g8, u8 = qa.gated_fwd(w[0], w[1], 40, 4, e8, e32, e8, e32, 0, 4, 256, act8=True)
    assert h.shape == (40, 0) and qa.gated_bwd(h, g8, u8).shape == (40, 0)


BWD_SHAPES = [(1, 1), (1, 5632), (3, 40), (17, 33), (64, 1001), (130, 264), (1000, 96), (5, 70001)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,cols", BWD_SHAPES)
def test_backward(dev, rows, cols, act, dtype):
    log(f"backward {rows}x{cols} {act} {dtype}")
    gen = torch.Generator().manual_seed(rows + cols)
    g, u = (torch.randn((rows, cols), generator=gen) * 2 for _ in range(2))
    g[:, ::17] *= 10
    dh = (1e-3 * torch.randn((rows, cols), generator=gen)).to(dtype)
    g8, u8 = qa.act8_save(g.to(dev)), qa.act8_save(u.to(dev))
    got = qa.gated_bwd(dh.to(dev), g8, u8, act=act)
    want, err = fo.gated_bwd(fo.f64(dh), fo.act8(fo.f64(g))[2], fo.act8(fo.f64(u))[2], act)
    r = fo.check("dgu", got, want, err + 2.0 ** -126)
    log(f"error / tolerance {r:.3g}")


def test_backward_of_bad_blocks(dev):
    """A block of a checkpoint that stood for NaN gives NaN there and nowhere else."""
    log("NaN blocks")
    gen = torch.Generator().manual_seed(3)
    g, u = (torch.randn((4, 96), generator=gen) for _ in range(2))
    g[1, 40] = float("nan")
    dh = torch.randn((4, 96), generator=gen).to(dev)
    out = qa.gated_bwd(dh, qa.act8_save(g.to(dev)), qa.act8_save(u.to(dev)))
    bad = torch.zeros((4, 192), dtype=torch.bool)
    bad[1, 32:64] = bad[1, 96 + 32:96 + 64] = True
    assert torch.equal(torch.isnan(out).cpu(), bad)


def test_backward_against_differences(dev):
    """Both gradients against central differences of act(g) u in 64 bits."""
    log("differences")
    gen = torch.Generator().manual_seed(4)
    for act in ("silu", "gelu"):
        g, u, dh = (torch.randn((5, 64), generator=gen) for _ in range(3))
        g8, u8 = qa.act8_save(g.to(dev)), qa.act8_save(u.to(dev))
        got = fo.f64(qa.gated_bwd(dh.to(dev), g8, u8, act=act))
        gv, uv, d = fo.act8(fo.f64(g))[2], fo.act8(fo.f64(u))[2], fo.f64(dh)
        s = 1e-4
        diff = (fo.act(gv + s, act)[0] - fo.act(gv - s, act)[0]) / (2 * s) * uv * d
        # s^2 / 6 |act'''| < 2 s^2 / 6, and the fp32 result's few roundings
        tol = (2 * s * s / 6 + 64 * fo.U) * np.abs(uv * d) + 1e-12
        assert (np.abs(got[:, :64] - diff) <= tol).all()
        assert (np.abs(got[:, 64:] - fo.act(gv, act)[0] * d) <= 64 * fo.U * np.abs(d)).all()


def test_other_stream(dev):
    log("other stream")
    n, k, m = 300, 512, 256
    ops = case(dev, n, k, m, 4, 4)
    want = call(ops, n, k, m, 4, 4, act8=True)
    dh = torch.randn((n, m), device=dev).to(torch.bfloat16)
    want_b = qa.gated_bwd(dh, want[1], want[2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(ops, n, k, m, 4, 4, act8=True, stream=side)
    got_b = qa.gated_bwd(dh, got[1], got[2], stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want_b, got_b)


def test_large_offsets(dev):
    """More than 2^31 outputs (2^32 bytes of them): the last rows as a call on those rows alone gives them."""
    n, k, m = (1 << 31) // 8192 + 96, 128, 8192
    log(f"{n}x{k}x{m}")
    x = torch.randn((n, k), device=dev).to(torch.bfloat16)
    _, xs, _, xo = qa.quantize_fwd_op(x, 128, 4)
    _, ts, _, to = qa.quantize_fwd_op(x[-96:].contiguous(), 128, 4)
    w = [qa.quantize_fwd_op(torch.randn((m, k), device=dev).to(torch.bfloat16), 128, 4) for _ in range(2)]
    args = (w[0][3], w[0][1], w[1][3], w[1][1], m, 4, k)
    h, g8, u8 = qa.gated_fwd(xo, xs, n, 4, *args, act8=True)
    th, tg, tu = qa.gated_fwd(to, ts, 96, 4, *args, act8=True)
    assert torch.equal(h[-96:], th)
    for a, c in zip((*g8, *u8), (*tg, *tu)):
        assert torch.equal(a[-96:], c)
    out = qa.gated_bwd(h, g8, u8)
    assert torch.equal(out[-96:], qa.gated_bwd(th, tg, tu))


def test_largest_k(dev):
    """k = 32768 columns, the widest row the quantiser writes: the sums stay exact."""
    n, k, m = 70, 32768, 64
    log(f"{n}x{k}x{m}")
    ops = case(dev, n, k, m, 4, 4)
    for rows in (n, 20):
        (xo, xs, lx) = quantised(dev, rows, k, 4, 1)
        want, _, _, err, _, _ = fo.gated_fwd(lx, ops[1][2], ops[2][2], "silu")
        h, _, _ = call(((xo, xs, lx), ops[1], ops[2]), rows, k, m, 4, 4, out_dtype=torch.float32)
        fo.check("h", h, want, err)
