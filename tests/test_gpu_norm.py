"""Layer norm's kernels against the definition in 64 bits, with bounds that count fp32 roundings."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import feedforward_oracle as fo
import quantization_aware_amd as qa

pytestmark = pytest.mark.gpu
EPS = 1e-5


def log(msg: str) -> None:
    print(f"[gpu-norm] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    return torch.device("cuda", 0)


SHAPES = [(1, 1), (5, 2), (1, 2048), (3, 7), (64, 31), (9, 32), (130, 100), (2050, 64), (33, 512), (40, 513), (7, 1000),
          (65, 1111), (18, 2048), (6, 2056), (5, 2049), (9, 4096), (4, 5632), (3, 8192), (3, 8200), (2, 9001),
          (3, 16384), (2, 16392), (5, 20001), (3, 32768), (600, 96), (515, 1000), (1030, 640), (520, 2048), (513, 1111)]


def inputs(rows, cols, dtype, pdtype, seed, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) + offset
    if cols >= 100:
        x[:, 5::100] *= 20
    x = x.to(dtype)
    dy = (torch.randn((rows, cols), generator=g) * 1e-2).to(dtype)
    w = (1 + 0.2 * torch.randn((cols,), generator=g)).to(pdtype)
    b = (0.2 * torch.randn((cols,), generator=g)).to(pdtype)
    return x, dy, w, b


def run_fwd(dev, x, w, b, act8=False):
    out = qa.layer_norm_fwd(x.to(dev), None if w is None else w.to(dev), None if b is None else b.to(dev), EPS,
                            act8=act8)
    return out


def check_fwd(out, x, w, b):
    y, mean, rstd, kept = out
    x64 = fo.f64(x)
    w64, b64 = (None if t is None else fo.f64(t) for t in (w, b))
    wy, wm, wr, wx = fo.norm_fwd(x64, w64, b64, EPS)
    ey, em, er, ex = fo.norm_fwd_bounds(x64, w64, b64, EPS)
    r = [fo.check("y", y, wy, ey), fo.check("mean", mean, wm, em), fo.check("rstd", rstd, wr, er)]
    if kept is not None:
        fo.check_act8_of(kept[0].cpu().numpy(), kept[1].cpu().numpy(), wx, ex)
    return r


@pytest.mark.parametrize("dtype,pdtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(dev, rows, cols, dtype, pdtype):
    log(f"forward {rows}x{cols} {dtype}")
    x, _, w, b = inputs(rows, cols, dtype, pdtype, rows + 31 * cols)
    r = check_fwd(run_fwd(dev, x, w, b, act8=True), x, w, b)
    log(f"error / tolerance {max(r):.3g}")
    plain = run_fwd(dev, x, w, b)
    kept = run_fwd(dev, x, w, b, act8=True)
    assert plain[3] is None
    for i in range(3):
        assert torch.equal(plain[i], kept[i])


@pytest.mark.parametrize("which", ["none", "weight", "bias"])
def test_forward_without_parameters(dev, which):
    log(f"parameters: {which}")
    x, _, w, b = inputs(20, 1000, torch.bfloat16, torch.bfloat16, 3)
    w, b = (w if which == "weight" else None), (b if which == "bias" else None)
    check_fwd(run_fwd(dev, x, w, b, act8=True), x, w, b)


@pytest.mark.parametrize("dtype,pdtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("act8", [False, True])
def test_backward(dev, rows, cols, dtype, pdtype, act8):
    log(f"backward {rows}x{cols} {dtype} act8={act8}")
    x, dy, w, b = inputs(rows, cols, dtype, pdtype, rows + 37 * cols)
    _, mean, rstd, kept = run_fwd(dev, x, w, b, act8=act8)
    if act8:
        xhat = fo.act8_values(kept[0].cpu().numpy(), kept[1].cpu().numpy())
        src = dict(act8=kept)
    else:
        xhat = (fo.f64(x) - fo.f64(mean)[:, None]) * fo.f64(rstd)[:, None]
        src = dict(x=x.to(dev), mean=mean)
    got = qa.layer_norm_bwd(dy.to(dev), rstd, w.to(dev), bias_grad=True, **src)
    args = (fo.f64(dy), xhat, fo.f64(rstd), fo.f64(w))
    ratios = [fo.check(n, g, want, err) for n, g, want, err in
              zip(("dx", "dw", "db"), got, fo.norm_bwd(*args), fo.norm_bwd_bounds(*args))]
    assert got[1].dtype == pdtype and got[2].dtype == pdtype
    log(f"error / tolerance {max(ratios):.3g}")
    # the same call again, and each gradient alone, give the same bits
    again = qa.layer_norm_bwd(dy.to(dev), rstd, w.to(dev), bias_grad=True, **src)
    for a, c in zip(got, again):
        assert torch.equal(a, c)
    only = qa.layer_norm_bwd(dy.to(dev), rstd, w.to(dev), weight_grad=False, **src)
    assert only[1] is None and only[2] is None
    fo.check("dx alone", only[0], fo.norm_bwd(*args)[0], fo.norm_bwd_bounds(*args)[0])
    only = qa.layer_norm_bwd(dy.to(dev), rstd, w.to(dev), input_grad=False, **src)
    assert only[0] is None and only[2] is None and torch.equal(only[1], got[1])


def test_backward_without_weight(dev):
    log("no weight")
    x, dy, _, _ = inputs(50, 640, torch.bfloat16, torch.float32, 8)
    _, mean, rstd, _ = run_fwd(dev, x, None, None)
    xhat = (fo.f64(x) - fo.f64(mean)[:, None]) * fo.f64(rstd)[:, None]
    dx, dw, db = qa.layer_norm_bwd(dy.to(dev), rstd, x=x.to(dev), mean=mean, bias_grad=True)
    args = (fo.f64(dy), xhat, fo.f64(rstd), None)
    assert dw is None and db.dtype == torch.float32
    fo.check("dx", dx, fo.norm_bwd(*args)[0], fo.norm_bwd_bounds(*args)[0])
    fo.check("db", db, fo.norm_bwd(*args)[2], fo.norm_bwd_bounds(*args)[2])


@pytest.mark.parametrize("rows,cols", [(8193, 1111), (8200, 1032), (4097, 1500), (2049, 600), (1025, 2049), (300, 5631)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_past_the_few(dev, rows, cols, dtype):
    """Either side of the numbers of rows at which rows are given to fewer threads, or sums to fewer workgroups."""
    test_forward(dev, rows, cols, dtype, torch.float32)
    test_backward(dev, rows, cols, dtype, torch.float32, False)
    test_backward(dev, rows, cols, dtype, torch.bfloat16, True)


def test_many_rows(dev):
    """More rows than workgroups walk at once, few columns."""
    log("300000x24")
    x, dy, w, b = inputs(300000, 24, torch.bfloat16, torch.float32, 12)
    out = run_fwd(dev, x, w, b)
    check_fwd(out, x, w, b)
    xhat = (fo.f64(x) - fo.f64(out[1])[:, None]) * fo.f64(out[2])[:, None]
    got = qa.layer_norm_bwd(dy.to(dev), out[2], w.to(dev), x=x.to(dev), mean=out[1], bias_grad=True)
    args = (fo.f64(dy), xhat, fo.f64(out[2]), fo.f64(w))
    for n, g, want, err in zip(("dx", "dw", "db"), got, fo.norm_bwd(*args), fo.norm_bwd_bounds(*args)):
        fo.check(n, g, want, err)


def test_large_offset_keeps_its_digits(dev):
    """A common offset 1000 times the spread costs the mean's rounding, not the variance."""
    log("offset 1000")
    x, _, w, b = inputs(40, 2048, torch.float32, torch.float32, 21, offset=1000.0)
    check_fwd(run_fwd(dev, x, w, b), x, w, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(64, 100), (40, 500), (100, 1111), (300, 1000), (64, 2048), (9000, 2048), (9000, 1111),
                                       (40, 4096), (33, 5631), (9, 16384), (5, 20001)])
def test_mean_of_an_exact_sum(dev, rows, cols, dtype):
    """Entries of a coarse grid, whose fp32 sum is exact in any order (whole multiples of 2^-6 below 2^17): the first
    sum gives the mean correctly rounded, and the roundings of x - mean are not taken for a part of it.  They are at
    most U |x - mean| each, U a quarter to a half of the entries' rms on average here; the sum's own rounding adds
    about U rms (64 / cols)^(1/2) or less."""
    log(f"exact sums {rows}x{cols} {dtype}")
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn((rows, cols), generator=g) + 0.1
    x[:, 5::100] *= 16
    x = (torch.round(x * 64) / 64).to(dtype)
    x64 = fo.f64(x)
    assert np.abs(x64).sum(axis=1).max() < 2 ** 17
    _, mean, _, _ = run_fwd(dev, x, None, None)
    want = (x64.sum(axis=1) / cols).astype(np.float32)
    off = (mean.cpu().numpy() != want)
    assert not off.any(), f"{off.sum()} of {rows} means are not the correctly rounded ones"


def test_constant_and_zero_rows(dev):
    log("constant rows")
    x = torch.zeros((4, 257))
    x[1], x[2], x[3, 5] = 3.5, -1e4, 1.0
    out = run_fwd(dev, x, None, None, act8=True)
    assert torch.equal(out[0][:3].cpu(), torch.zeros((3, 257)))
    check_fwd((out[0][3:], out[1][3:], out[2][3:], None), x[3:], None, None)
    assert np.allclose(fo.f64(out[2][:3]), EPS ** -0.5, rtol=4 * fo.U * 2, atol=0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_entries_stay_in_their_row(dev, bad):
    log(f"{bad}")
    x, dy, w, b = inputs(9, 700, torch.bfloat16, torch.float32, 6)
    clean = run_fwd(dev, x, w, b, act8=True)
    broken = x.clone()
    broken[4, 17] = bad
    got = run_fwd(dev, broken, w, b, act8=True)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    for i in range(3):
        assert torch.equal(clean[i][keep], got[i][keep])
    assert torch.equal(clean[3][0][keep], got[3][0][keep])
    assert torch.isnan(got[0][4]).all()
    assert (got[3][1][4] == 255).all()  # the checkpoint stands for NaN too
    dx, _, _ = qa.layer_norm_bwd(dy.to(dev), got[2], w.to(dev), act8=got[3])
    assert torch.isnan(dx[4]).all() and torch.isfinite(dx[keep]).all()


@pytest.mark.parametrize("cols", [7, 19, 33, 100, 257, 700, 993, 1000, 1111, 2049, 5640, 9001, 16392, 20001])
def test_checkpoint_is_that_of_the_normalised_input(dev, cols):
    """Without parameters an fp32 y is xhat itself, so the checkpoint is the one that saving y gives, byte for byte:
    rows of one value (zeros), and rows whose last block holds next to nothing, among them."""
    log(f"checkpoint of {cols} columns")
    g = torch.Generator().manual_seed(cols)
    for rows in (6, 600):
        x = torch.randn((rows, cols), generator=g) + 1000.3
        x[0], x[1] = 0.1, -1e4 / 3
        tail = cols - (cols - 1) // 32 * 32
        x[2:4, -tail:] = x[2:4].mean(1, keepdim=True)
        y, _, _, kept = run_fwd(dev, x, None, None, act8=True)
        want = qa.act8_save(y)
        assert torch.equal(kept[1], want[1]) and torch.equal(kept[0], want[0])


@pytest.mark.parametrize("cols", [19, 700, 1111, 9001])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_statistics_of_bad_rows(dev, cols, bad):
    """A row with an infinity or NaN has no finite statistics, wherever it lies."""
    log(f"{bad} in {cols} columns")
    for at in (0, cols - 1):
        x, _, w, b = inputs(5, cols, torch.float32, torch.float32, 8)
        x[2, at] = bad
        y, mean, rstd, _ = run_fwd(dev, x, w, b)
        assert torch.isnan(y[2]).all() and torch.isnan(rstd[2]) and not torch.isfinite(mean[2])
        keep = [0, 1, 3, 4]
        assert torch.isfinite(y[keep]).all() and torch.isfinite(rstd[keep]).all()


@pytest.mark.parametrize("cols", [19, 700, 2048, 9001])
def test_rows_whose_sum_overflows(dev, cols):
    """Finite entries whose fp32 sum is none: no finite statistics either."""
    log(f"overflow in {cols} columns")
    for big in (3e38, -3e38):
        x, _, w, b = inputs(5, cols, torch.float32, torch.float32, 9)
        x[2] = big
        y, mean, rstd, _ = run_fwd(dev, x, w, b)
        assert torch.isnan(y[2]).all() and torch.isnan(rstd[2]) and not torch.isfinite(mean[2])
        keep = [0, 1, 3, 4]
        assert torch.isfinite(y[keep]).all() and torch.isfinite(rstd[keep]).all()


def test_no_rows(dev):
    log("no rows")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    y, mean, rstd, kept = qa.layer_norm_fwd(x, w, w, EPS, act8=True)
    assert y.shape == (0, 64)
    dx, dw, db = qa.layer_norm_bwd(y, rstd, w, act8=kept, bias_grad=True)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_gradient_against_differences(dev):
    """dx, dw and db against central differences of the forward, in fp32."""
    log("differences")
    x, dy, w, b = inputs(4, 48, torch.float32, torch.float32, 77)
    _, mean, rstd, _ = run_fwd(dev, x, w, b)
    dx, dw, db = qa.layer_norm_bwd(dy.to(dev), rstd, w.to(dev), x=x.to(dev), mean=mean, bias_grad=True)
    g = torch.Generator().manual_seed(78)
    h = 2.0 ** -7
    for name, grad, base in (("x", dx, x), ("w", dw, w), ("b", db, b)):
        d = torch.randn(base.shape, generator=g)
        d /= d.abs().max()
        vals = []
        for s in (h, -h):
            p = {"x": x, "w": w, "b": b}
            p[name] = base + s * d
            vals.append(fo.f64(run_fwd(dev, p["x"], p["w"], p["b"])[0]))
        diff = ((vals[0] - vals[1]) * fo.f64(dy)).sum() / (2 * h)
        an = (fo.f64(grad) * fo.f64(d)).sum()
        # fp32 forward errors of about 4 U |y| over 2 h, and the curvature h^2 / 6 |y'''| with |y'''| of order 10 / row
        tol = (8 * fo.U / (2 * h) * (1 + np.abs(vals[0])) + h * h * 10).ravel() @ np.abs(fo.f64(dy)).ravel()
        assert abs(diff - an) <= tol, (name, diff, an, tol)


def test_other_stream(dev):
    log("other stream")
    x, dy, w, b = inputs(3000, 1024, torch.bfloat16, torch.float32, 14)
    x, dy, w, b = (t.to(dev) for t in (x, dy, w, b))
    want = qa.layer_norm_fwd(x, w, b, EPS)
    want_g = qa.layer_norm_bwd(dy, want[2], w, x=x, mean=want[1], bias_grad=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = qa.layer_norm_fwd(x, w, b, EPS, stream=side)
    got_g = qa.layer_norm_bwd(dy, got[2], w, x=x, mean=got[1], bias_grad=True, stream=side)
    junk = [torch.full((1 << 22,), 3.0, device=dev) for _ in range(4)]  # would land in a workspace given back early
    side.synchronize()
    del junk
    for a, c in zip((*want[:3], *want_g), (*got[:3], *got_g)):
        assert torch.equal(a, c)


def test_large_offsets(dev):
    """More than 2^31 entries (2^32 bytes): the last rows, and the columns' sums of a gradient that is zero before them."""
    rows, cols = (1 << 31) // 2048 + 64, 2048
    log(f"{rows}x{cols}")
    x = torch.randn((rows, cols), device=dev).to(torch.bfloat16)
    w = torch.randn((cols,), device=dev)
    y, mean, rstd, kept = qa.layer_norm_fwd(x, w, w, EPS, act8=True)
    tail = x[-64:].contiguous()
    ty, tmean, trstd, tkept = qa.layer_norm_fwd(tail, w, w, EPS, act8=True)
    # (rows of a large call are a wave's, of a small one a workgroup's: the sums' orders differ)
    assert torch.allclose(y[-64:].float(), ty.float(), rtol=2 ** -7, atol=1e-5)
    assert torch.allclose(rstd[-64:], trstd, rtol=2e-6, atol=0)
    check_fwd((y[-64:], mean[-64:], rstd[-64:], tuple(t[-64:] for t in kept)), tail, w, w)
    dy = torch.zeros_like(x)
    dy[-64:] = torch.randn((64, cols), device=dev).to(torch.bfloat16)
    for src in (dict(act8=kept), dict(x=x, mean=mean)):
        got = qa.layer_norm_bwd(dy, rstd, w, bias_grad=True, **src)
        assert not got[0][:-64].any()
        if "x" in src:
            xhat = (fo.f64(tail) - fo.f64(mean[-64:])[:, None]) * fo.f64(rstd[-64:])[:, None]
        else:
            xhat = fo.act8_values(*(t[-64:].cpu().numpy() for t in kept))
        args = (fo.f64(dy[-64:]), xhat, fo.f64(rstd[-64:]), fo.f64(w))
        for name, g, want, err in zip(("dx", "dw", "db"), (got[0][-64:], *got[1:]), fo.norm_bwd(*args),
                                      fo.norm_bwd_bounds(*args)):
            fo.check(name, g, want, err)
