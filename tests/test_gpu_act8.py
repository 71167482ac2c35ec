"""Activation checkpoints in 8 bits against their definition: every byte has to be equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import feedforward_oracle as fo
import quantization_aware_amd as qa

pytestmark = pytest.mark.gpu


def log(msg: str) -> None:
    print(f"[gpu-act8] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    return torch.device("cuda", 0)


def make(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(3 * torch.randn((rows, 1), generator=g))
    if cols > 3:
        x[:, 3::50] *= 20
    return x.to(dtype)


def check(x, dev):
    codes, scale = qa.act8_save(x.to(dev))
    want_c, want_s, want_v = fo.act8(fo.f64(x))
    assert np.array_equal(scale.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    for dt in (torch.bfloat16, torch.float32):
        out = qa.act8_load(codes, scale, out_dtype=dt)
        assert np.array_equal(fo.f64(out), want_v, equal_nan=True), dt
    return codes, scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 31), (4, 32), (7, 33), (1, 2048), (33, 64), (129, 96),
                                       (17, 1000), (10, 1001), (3, 5632), (1025, 8), (2, 40000), (2000, 1), (0, 64)])
def test_bytes(dev, rows, cols, dtype):
    log(f"{rows}x{cols} {dtype}")
    check(make(rows, cols, dtype, rows * 7919 + cols), dev)


@pytest.mark.parametrize("cols", [64, 45])
def test_special_values(dev, cols):
    """Zero blocks, subnormals, the largest numbers, ties, the clamp, infinities and NaN."""
    log(f"special values, {cols} columns")
    rows = []
    z = torch.zeros(cols)
    rows.append(z.clone())
    for v in (2.0 ** -149, 2.0 ** -133, 1.5 * 2.0 ** -127, 2.0 ** -126, 3.4028234e38, 1.0, 1.9999999, 127.5 / 64,
              -127.49999 / 64):
        r = z.clone()
        r[1] = v
        r[2] = -v / 2
        r[3] = v * 0.37
        rows.append(r)
    r = z.clone()  # ties at every half step below 1.0
    r[0] = 1.0
    n = min(cols - 1, 40)
    r[1:1 + n] = (torch.arange(n) + 0.5) / 64
    rows.append(r)
    for bad in (float("inf"), float("-inf"), float("nan")):
        r = torch.linspace(-1, 1, cols)
        r[cols - 1] = bad
        rows.append(r)
        r = torch.linspace(-1, 1, cols)
        r[0] = bad
        rows.append(r)
    check(torch.stack(rows).float(), dev)


def test_second_save_gives_the_same_bytes(dev):
    log("idempotent")
    codes, scale = check(make(64, 416, torch.float32, 5), dev)
    for dt in (torch.bfloat16, torch.float32):
        again = qa.act8_save(qa.act8_load(codes, scale, out_dtype=dt))
        assert torch.equal(again[0], codes) and torch.equal(again[1], scale)


def test_large_offsets(dev):
    """Entries past 2^31 bytes of the codes and 2^32 of the tensor."""
    rows, cols = (1 << 31) // 4096 + 3, 4096
    log(f"{rows}x{cols} bf16")
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=dev)
    tail = make(8, cols, torch.bfloat16, 9)
    x[-8:] = tail.to(dev)
    codes, scale = qa.act8_save(x)
    c, s, v = fo.act8(fo.f64(tail))
    assert np.array_equal(codes[-8:].cpu().numpy(), c) and np.array_equal(scale[-8:].cpu().numpy(), s)
    assert int(codes[:-8].amax()) == 0
    out = qa.act8_load(codes, scale, out=x)
    assert np.array_equal(fo.f64(out[-8:]), v)


def test_other_stream_and_caller_buffers(dev):
    log("other stream")
    x = make(257, 320, torch.bfloat16, 11).to(dev)
    side = torch.cuda.Stream()
    codes = torch.full((257, 320), 7, dtype=torch.int8, device=dev)
    scale = torch.full((257, 10), 7, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    got = qa.act8_save(x, codes=codes, scale=scale, stream=side)
    out = torch.empty((257, 320), dtype=torch.float32, device=dev)
    qa.act8_load(*got, out=out, stream=side)
    side.synchronize()
    assert got[0] is codes and got[1] is scale
    assert np.array_equal(fo.f64(out), fo.act8(fo.f64(x))[2])
