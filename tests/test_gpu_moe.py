"""The mixture-of-experts layer for a few tokens against its definition in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import moe_oracle as mo
import quantization_aware_amd as qa

pytestmark = pytest.mark.gpu


def log(msg: str) -> None:
    print(f"[gpu-moe] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    return torch.device("cuda", 0)


def coded(shape, bits, gen, std=1.0):
    half = 2 ** (bits - 1)
    c = torch.floor(torch.randn(shape, generator=gen) * half / 2.5).clamp(-half, half - 1).to(torch.int8)
    return c, std * torch.exp(0.25 * torch.randn(shape[:-1], generator=gen))


class Layer:
    """An expert layer's codes and scales, packed where asked, and its values in 64 bits."""

    def __init__(self, dev, e, k, m, bits, packed, seed):
        g = torch.Generator().manual_seed(seed)
        self.bits, self.dev = bits, dev
        self.args, self.values = [], []
        for shape in ((e, m, k), (e, m, k), (e, k, m)):
            c, s = coded(shape, bits, g, 2.0 * shape[-1] ** -0.5)
            self.values.append(mo.values(c.numpy().astype(np.float64), s.numpy(), bits))
            if packed:
                u = (c + 8).to(torch.uint8)
                c = u[..., 0::2] | (u[..., 1::2] << 4)
            self.args += [c.to(dev), s.to(dev)]

    def __call__(self, x, xs, xb, logits, top, **kw):
        return qa.moe_fwd(x, xs, xb, logits, *self.args, self.bits, top, **kw)


def tokens(dev, n, k, bits, seed):
    g = torch.Generator().manual_seed(seed)
    c, s = coded((n, k), bits, g)
    return c.to(dev), s.to(dev), mo.values(c.numpy().astype(np.float64), s.numpy(), bits)


def run_case(dev, n, e, top, k, m, xb, wb, hb, block, act, packed, over_all=False, logits=None, out_dtype=torch.float32,
             seed=1):
    layer = Layer(dev, e, k, m, wb, packed, seed)
    x, xs, xv = tokens(dev, n, k, xb, seed + 1)
    if logits is None:
        logits = torch.randn((n, e), generator=torch.Generator().manual_seed(seed + 2))
    y = layer(x, xs, xb, logits.to(dev), top, block=block, h_bits=hb, act=act, over_all=over_all, out_dtype=out_dtype)
    want, bound = mo.moe(xv, logits.double().numpy(), *layer.values, top, block, hb, act, over_all)
    eps = torch.finfo(torch.bfloat16).eps / 2 if out_dtype == torch.bfloat16 else mo.U
    assert y.shape == (n, k) and y.dtype == out_dtype
    used = mo.check(y.double().cpu().numpy(), eps, want, bound)
    log(f"n={n} e={e} top={top} {k}x{m} b={xb},{wb},{hb} {act}: {used:.3g} of the bound")
    return layer, x, xs, logits.to(dev), y


CASES = [
    # n, e, top, k, m, x bits, weight bits, h bits, block, activation, packed
    (1, 1, 1, 64, 64, 8, 8, 8, 64, "silu", False),
    (1, 64, 8, 256, 128, 4, 4, 4, 128, "silu", True),
    (1, 256, 3, 128, 64, 8, 4, 8, 64, "gelu", True),
    (1, 5, 5, 320, 192, 8, 8, 4, 64, "gelu", False),
    (2, 130, 32, 128, 128, 5, 3, 6, 128, "silu", False),
    (3, 70, 7, 192, 256, 8, 4, 8, 256, "silu", True),
    (7, 13, 3, 704, 448, 6, 5, 6, 64, "gelu", False),
    (8, 65, 8, 64, 64, 1, 1, 1, 64, "silu", False),
    (16, 8, 2, 512, 320, 8, 4, 8, 64, "silu", True),
    (17, 2, 1, 192, 64, 8, 8, 8, 64, "silu", False),
    (33, 4, 2, 448, 1088, 8, 4, 4, 64, "gelu", True),
    (64, 3, 3, 128, 128, 8, 8, 8, 128, "gelu", False),
    (64, 20, 2, 2048, 256, 8, 8, 8, 256, "silu", False),
    (64, 100, 4, 64, 128, 2, 2, 2, 128, "silu", False),
    (1, 3, 2, 4160, 64, 8, 4, 8, 64, "silu", True),
    (5, 2, 2, 64, 8192, 8, 4, 8, 256, "silu", True),
    (20, 2, 2, 64, 8192, 8, 8, 8, 64, "gelu", False),
]


@pytest.mark.parametrize("over_all", [False, True])
@pytest.mark.parametrize("n,e,top,k,m,xb,wb,hb,block,act,packed", CASES)
def test_layer(dev, n, e, top, k, m, xb, wb, hb, block, act, packed, over_all):
    log(f"start n={n} e={e} top={top} {k}x{m} b={xb},{wb},{hb} block {block} {act} packed={packed}")
    run_case(dev, n, e, top, k, m, xb, wb, hb, block, act, packed, over_all, seed=n + e + k)


@pytest.mark.parametrize("packed", [False, True])
def test_output_and_logits_types(dev, packed):
    log("bf16 outputs and logits")
    args = (9, 12, 3, 256, 192, 8, 4, 8, 64, "silu", packed)
    _, _, _, logits, y32 = run_case(dev, *args)
    _, _, _, _, y16 = run_case(dev, *args, out_dtype=torch.bfloat16)
    assert torch.equal(y16, y32.to(torch.bfloat16))
    run_case(dev, *args, logits=torch.round(2 * torch.randn(9, 12, generator=torch.Generator().manual_seed(5))).to(
        torch.bfloat16))


@pytest.mark.parametrize("n,e,top", [(1, 64, 8), (6, 64, 4), (40, 64, 4), (40, 200, 6)])
def test_equal_logits_take_the_lowest(dev, n, e, top):
    log(f"ties n={n} e={e} top={top}")
    g = torch.Generator().manual_seed(3)
    logits = torch.randint(0, 3, (n, e), generator=g).float()
    logits[0] = 1.5
    logits[-1, ::2] = -0.0
    logits[-1, 1::2] = 0.0
    run_case(dev, n, e, top, 128, 64, 8, 8, 8, 64, "silu", False, logits=logits)


@pytest.mark.parametrize("n,e,top", [(5, 64, 8), (6, 8, 4), (40, 64, 4)])
@pytest.mark.parametrize("over_all", [False, True])
def test_masked_and_special_logits(dev, n, e, top, over_all):
    """Experts that are masked, tokens with fewer experts than top_k or none, NaN and +infinity."""
    log(f"masks n={n} e={e} top={top}")
    g = torch.Generator().manual_seed(4)
    logits = torch.randn((n, e), generator=g)
    logits[:, 3] = -float("inf")
    logits[0] = -float("inf")
    logits[1] = -float("inf")
    logits[1, e - 1] = -3e38
    logits[2, 2:] = -float("inf")
    logits[3, 1] = float("nan")
    logits[4, 0] = float("inf")
    _, _, _, _, y = run_case(dev, n, e, top, 128, 64, 8, 8, 8, 64, "silu", False, over_all, logits=logits)
    assert (y[0] == 0).all() and y[3].isnan().all() and y[4].isnan().all()


def test_one_expert_for_all_tokens(dev):
    logits = torch.randn((64, 16), generator=torch.Generator().manual_seed(6))
    logits[:, 5] = 10.0
    logits[:, 11] = 9.0
    run_case(dev, 64, 16, 2, 256, 128, 8, 4, 8, 128, "silu", True, logits=logits)


def test_tokens_stand_alone(dev):
    """A token's output does not depend on the others, bit for bit, nor on a second call."""
    layer, x, xs, logits, y = run_case(dev, 48, 24, 4, 512, 256, 8, 4, 8, 128, "silu", True)
    for t in (0, 7, 47):
        one = layer(x[t:t + 1].clone(), xs[t:t + 1].clone(), 8, logits[t:t + 1].clone(), 4, block=128, h_bits=8,
                    out_dtype=torch.float32)
        assert torch.equal(one[0], y[t])
    assert torch.equal(y, layer(x, xs, 8, logits, 4, block=128, h_bits=8, out_dtype=torch.float32))


def test_rows_behind_the_last_are_left(dev):
    layer = Layer(dev, 6, 192, 128, 8, False, 9)
    x, xs, _ = tokens(dev, 5, 192, 8, 10)
    logits = torch.randn(5, 6, device=dev)
    buf = torch.full((9, 192), 7.0, dtype=torch.bfloat16, device=dev)
    y = layer(x, xs, 8, logits, 2, out=buf[:5])
    assert (buf[5:] == 7.0).all() and y.data_ptr() == buf.data_ptr()
    assert torch.equal(y, layer(x, xs, 8, logits, 2))
    assert layer(x[:0], xs[:0], 8, logits[:0], 2).shape == (0, 192)


def test_zero_hidden_rows(dev):
    """A token whose h is zero for an expert (scale 0) gets nothing from it."""
    layer = Layer(dev, 3, 128, 64, 8, False, 11)
    layer.args[3][1] = 0.0  # expert 1's up scales
    x, xs, _ = tokens(dev, 4, 128, 8, 12)
    logits = torch.tensor([[0.0, 50.0, -50.0]] * 4, device=dev)
    y = layer(x, xs, 8, logits, 1, block=64, out_dtype=torch.float32)
    assert (y == 0).all()


def test_past_32_bit_offsets(dev):
    """Weights of more than 2^32 bytes."""
    e, k, m = 40, 32768, 4096
    log("experts of 5 GB")
    g = torch.Generator().manual_seed(13)
    small = [coded(s, 4, g) for s in ((m, k), (m, k), (k, m))]
    packed = []
    for c, s in small:
        u = (c + 8).to(torch.uint8)
        packed.append(((u[:, 0::2] | (u[:, 1::2] << 4)).to(dev), s.to(dev)))
    x, xs, _ = tokens(dev, 3, k, 8, 14)
    alone = [t[None].contiguous() for pair in packed for t in pair]
    want = qa.moe_fwd(x, xs, 8, torch.zeros(3, 1, device=dev), *alone, 4, 1)
    args = []
    for w, s in packed:
        wide = torch.zeros((e, *w.shape), dtype=torch.uint8, device=dev)
        scale = torch.ones((e, *s.shape), device=dev)
        wide[-1], scale[-1] = w, s
        args += [wide, scale]
    logits = torch.zeros(3, e, device=dev)
    logits[:, -1] = 5.0
    assert torch.equal(want, qa.moe_fwd(x, xs, 8, logits, *args, 4, 1))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("n", [1, 4])
def test_few_tokens_with_some_experts_of_many(dev, n, packed):
    """Of top_k = 32 as many as are not masked: 17, 9, 1 and 32."""
    log(f"masked ranks n={n} packed={packed}")
    logits = torch.randn((n, 40), generator=torch.Generator().manual_seed(15))
    for t, found in enumerate((17, 9, 1)[:n]):
        logits[t, found:] = -float("inf")
    for over_all in (False, True):
        run_case(dev, n, 40, 32, 192, 320, 8, 4, 8, 64, "gelu", packed, over_all, logits=logits)


@pytest.mark.parametrize("n,top,m,e,packed", [(4, 8, 8192, 9, True), (3, 32, 2048, 33, False), (4, 9, 7296, 9, False),
                                              (4, 1, 8192, 2, False), (2, 6, 1088, 129, True)])
def test_few_tokens_as_among_many(dev, n, top, m, e, packed):
    """A few tokens' outputs are those they have in a larger batch, at the widths where the form changes."""
    log(f"few as many n={n} top={top} m={m}")
    layer, x, xs, logits, y = run_case(dev, 7, e, top, 128, m, 8, 4, 8, 64, "silu", packed, seed=n + m)
    few = layer(x[:n].clone(), xs[:n].clone(), 8, logits[:n].clone(), top, block=64, h_bits=8, out_dtype=torch.float32)
    assert torch.equal(few, y[:n])


@pytest.mark.parametrize("n,e,top,k,m,xb,wb,hb,block,act,packed", [
    # many tokens of few experts, few tokens of many, odd lengths and every type of code
    (35, 1, 1, 64, 64, 8, 8, 8, 64, "silu", False),
    (40, 64, 8, 256, 128, 4, 4, 4, 128, "silu", True),
    (33, 256, 3, 128, 64, 8, 4, 8, 64, "gelu", True),
    (47, 5, 5, 320, 192, 8, 8, 4, 64, "gelu", False),
    (34, 130, 32, 128, 128, 5, 3, 6, 128, "silu", False),
    (51, 70, 7, 192, 256, 8, 4, 8, 256, "silu", True),
    (39, 13, 3, 704, 448, 6, 5, 6, 64, "gelu", False),
    (64, 65, 8, 64, 64, 1, 1, 1, 64, "silu", False),
    (48, 8, 2, 512, 320, 8, 4, 8, 64, "silu", True),
    (36, 3, 2, 4160, 64, 8, 4, 8, 64, "silu", True),
    (37, 2, 2, 64, 8192, 8, 4, 8, 256, "silu", True),
    (64, 2, 2, 64, 8192, 8, 8, 8, 64, "gelu", False),
    (1, 33, 32, 64, 2112, 8, 4, 8, 64, "silu", True),
    (3, 9, 9, 64, 8192, 8, 4, 8, 128, "gelu", True),
    (5, 12, 9, 128, 7424, 8, 8, 8, 256, "silu", False),
])
def test_larger_batches_and_layers(dev, n, e, top, k, m, xb, wb, hb, block, act, packed):
    log(f"start n={n} e={e} top={top} {k}x{m} b={xb},{wb},{hb} block {block} {act} packed={packed}")
    run_case(dev, n, e, top, k, m, xb, wb, hb, block, act, packed, n % 2 == 0, seed=n + e + k)


@pytest.mark.parametrize("n,e,top,packed", [(33, 8, 2, True), (64, 24, 4, False)])
def test_tokens_among_others(dev, n, e, top, packed):
    """A token's output alone, in a few and in a full batch: the same bits."""
    log(f"tokens among others n={n} e={e}")
    layer, x, xs, logits, y = run_case(dev, n, e, top, 320, 192, 8, 4, 6, 64, "gelu", packed)
    for first, count in ((0, 1), (5, 3), (n - 9, 9), (1, 32)):
        rows = slice(first, first + count)
        part = layer(x[rows].clone(), xs[rows].clone(), 8, logits[rows].clone(), top, block=64, h_bits=6, act="gelu",
                     out_dtype=torch.float32)
        assert torch.equal(part, y[rows])


def test_past_32_bit_offsets_of_many_tokens(dev):
    """Weights of more than 2^32 bytes in a batch whose tokens share experts."""
    e, k, m, n = 40, 32768, 4096, 40
    log("experts of 5 GB, many tokens")
    g = torch.Generator().manual_seed(16)
    alone = []
    for shape in ((m, k), (m, k), (k, m)):
        c, s = coded(shape, 4, g)
        u = (c + 8).to(torch.uint8)
        alone += [(u[:, 0::2] | (u[:, 1::2] << 4)).to(dev)[None].contiguous(), s.to(dev)[None].contiguous()]
    x, xs, _ = tokens(dev, n, k, 8, 17)
    want = qa.moe_fwd(x, xs, 8, torch.zeros(n, 1, device=dev), *alone, 4, 1)
    args = []
    for t in alone:
        wide = torch.zeros((e, *t.shape[1:]), dtype=t.dtype, device=dev)
        wide[-1] = t[0]
        args.append(wide)
    logits = torch.zeros(n, e, device=dev)
    logits[:, -1] = 5.0
    assert torch.equal(want, qa.moe_fwd(x, xs, 8, logits, *args, 4, 1))


def test_on_a_stream_of_its_own(dev):
    """Calls with stream=, a few and many tokens at once on two streams, and no others waiting for them."""
    layer = Layer(dev, 16, 512, 256, 4, True, 18)
    sets = [tokens(dev, n, 512, 8, 19 + n)[:2] + (torch.randn(n, 16, device=dev),) for n in (2, 50)]
    want = [layer(x, xs, 8, logits, 4) for x, xs, logits in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[layer(x, xs, 8, logits, 4, stream=s) for (x, xs, logits), s in zip(sets, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(a, b) for a, b in zip(pair, want))
