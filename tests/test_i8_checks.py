"""Argument checks of the byte-code quantiser, the 8-bit integer product, the expert layer and their modules, on the CPU.

No call launches a kernel: the C entries get arguments that they must reject
before touching a buffer (the pointers are never dereferenced) or empty sizes,
and the binding gets CPU tensors, whose sizes and types it checks before their
device.
"""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch

import moe_oracle as mo
import quantization_aware_amd as qa
from quantization_aware_amd.experts import QuestMoE, route
from quantization_aware_amd.linear import QuestLinear, quest_linear

OK, EINVAL, EUNSUPPORTED, EALIGN = qa.QUEST_OK, qa.QUEST_EINVAL, qa.QUEST_EUNSUPPORTED, qa.QUEST_EALIGN
P = [0x100000000 * (i + 1) for i in range(16)]  # aligned and far apart


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qa.LIB_PATH):
        pytest.fail("libquest.so is not built; run `python -m quantization_aware_amd.build`")
    return qa.load_library()


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def i8(*shape):
    return t(*shape, dtype=torch.int8)


# ---------------------------------------------------------------------------
# The C entries
# ---------------------------------------------------------------------------

def quant(lib, x=P[0], dt=qa.QUEST_BF16, rows=4, cols=256, block=128, b=8, trust=1.0, codes=P[1], scale=P[2], mask=P[3]):
    return lib.quest_quantize_fwd_i8(x, dt, rows, cols, block, b, trust, codes, scale, mask, None)


def dequant(lib, codes=P[0], scale=P[1], rows=4, cols=192, b=8, out=P[2], dt=qa.QUEST_BF16):
    return lib.quest_dequantize_i8(codes, scale, rows, cols, b, out, dt, None)


def gemm(lib, a=P[0], sa=P[1], m=4, ab=8, b=P[2], sb=P[3], n=100, bb=8, k=192, out=P[4], dt=qa.QUEST_BF16):
    return lib.quest_gemm_i8(a, sa, m, ab, b, sb, n, bb, k, out, dt, None)


def moe(lib, x=P[0], xs=P[1], n=4, xb=8, logits=P[2], ldt=qa.QUEST_F32, e=8, top=2, over_all=0, g=P[3], gs=P[4], u=P[5],
        us=P[6], d=P[7], ds=P[8], wb=8, packed=0, k=192, m=256, block=128, hb=8, act=0, out=P[9], dt=qa.QUEST_BF16, ws=P[10]):
    return lib.quest_moe_fwd(x, xs, n, xb, logits, ldt, e, top, over_all, g, gs, u, us, d, ds, wb, packed, k, m, block, hb,
                             act, out, dt, ws, None)


def test_empty_calls_are_noops(lib):
    assert quant(lib, x=None, rows=0, codes=None, scale=None, mask=None) == OK
    assert dequant(lib, codes=None, scale=None, rows=0, out=None) == OK
    none = dict(a=None, sa=None, b=None, sb=None, out=None)
    assert gemm(lib, m=0, **none) == OK and gemm(lib, n=0, **none) == OK
    assert moe(lib, n=0, x=None, xs=None, logits=None, g=None, gs=None, u=None, us=None, d=None, ds=None, out=None,
               ws=None) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(block=96), EUNSUPPORTED), (dict(b=0), EUNSUPPORTED), (dict(b=9), EUNSUPPORTED), (dict(dt=7), EINVAL),
    (dict(trust=-1.0), EINVAL), (dict(trust=float("nan")), EINVAL), (dict(trust=float("inf")), EINVAL),
    (dict(rows=-1), EINVAL), (dict(cols=200), EINVAL), (dict(cols=0), EINVAL), (dict(cols=32896), EUNSUPPORTED),
    (dict(rows=1 << 40), EUNSUPPORTED), (dict(x=None), EINVAL), (dict(codes=None), EINVAL), (dict(scale=None), EINVAL),
    (dict(x=P[0] + 8), EALIGN), (dict(codes=P[1] + 1), EALIGN), (dict(scale=P[2] + 4), EALIGN), (dict(mask=P[3] + 2), EALIGN),
    (dict(codes=P[0] + 16), EINVAL), (dict(scale=P[1] + 1008), EINVAL), (dict(mask=P[2]), EINVAL),
])
def test_quantiser_rejects(lib, kw, status):
    assert quant(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(b=0), EUNSUPPORTED), (dict(b=9), EUNSUPPORTED), (dict(dt=-1), EINVAL), (dict(rows=-1), EINVAL),
    (dict(cols=100), EINVAL), (dict(cols=32832), EUNSUPPORTED), (dict(rows=1 << 40), EUNSUPPORTED), (dict(codes=None), EINVAL),
    (dict(scale=None), EINVAL), (dict(out=None), EINVAL), (dict(out=P[2] + 2), EALIGN), (dict(out=P[0] + 64), EINVAL),
    (dict(out=P[1]), EINVAL),
])
def test_dequantiser_rejects(lib, kw, status):
    assert dequant(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ab=0), EUNSUPPORTED), (dict(bb=9), EUNSUPPORTED), (dict(dt=3), EINVAL), (dict(m=-1), EINVAL), (dict(n=-1), EINVAL),
    (dict(k=0), EINVAL), (dict(k=-64), EINVAL), (dict(k=100), EUNSUPPORTED), (dict(k=32832), EUNSUPPORTED),
    (dict(n=(1 << 20) + 1), EUNSUPPORTED), (dict(m=(1 << 30) + 1), EUNSUPPORTED), (dict(m=1 << 30, n=1 << 20), EUNSUPPORTED),
    (dict(a=None), EINVAL), (dict(sa=None), EINVAL), (dict(b=None), EINVAL), (dict(sb=None), EINVAL), (dict(out=None), EINVAL),
    (dict(a=P[0] + 8), EALIGN), (dict(sa=P[1] + 4), EALIGN), (dict(b=P[2] + 1), EALIGN), (dict(sb=P[3] + 12), EALIGN),
    (dict(out=P[4] + 2), EALIGN), (dict(out=P[0] + 512), EINVAL), (dict(out=P[3]), EINVAL), (dict(out=P[2] - 16), EINVAL),
])
def test_product_rejects(lib, kw, status):
    assert gemm(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(block=32), EUNSUPPORTED), (dict(xb=0), EUNSUPPORTED), (dict(wb=9), EUNSUPPORTED), (dict(hb=0), EUNSUPPORTED),
    (dict(packed=1, wb=8), EUNSUPPORTED), (dict(packed=1, wb=3), EUNSUPPORTED), (dict(ldt=9), EINVAL), (dict(dt=9), EINVAL),
    (dict(act=2), EINVAL), (dict(n=-1), EINVAL), (dict(e=0), EINVAL), (dict(top=0), EINVAL), (dict(top=9), EINVAL),
    (dict(k=0), EINVAL), (dict(m=0), EINVAL), (dict(m=192), EINVAL), (dict(n=65), EUNSUPPORTED), (dict(e=257), EUNSUPPORTED),
    (dict(e=256, top=33), EUNSUPPORTED), (dict(k=200), EUNSUPPORTED), (dict(k=32832), EUNSUPPORTED), (dict(m=8320), EUNSUPPORTED),
    (dict(x=None), EINVAL), (dict(xs=None), EINVAL), (dict(logits=None), EINVAL), (dict(g=None), EINVAL), (dict(gs=None), EINVAL),
    (dict(u=None), EINVAL), (dict(us=None), EINVAL), (dict(d=None), EINVAL), (dict(ds=None), EINVAL), (dict(out=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(x=P[0] + 4), EALIGN), (dict(logits=P[2] + 4), EALIGN), (dict(ds=P[8] + 8), EALIGN),
    (dict(ws=P[10] + 8), EALIGN), (dict(out=P[0]), EINVAL), (dict(ws=P[9]), EINVAL), (dict(ws=P[3] - 64), EINVAL),
    (dict(out=P[8] + 128), EINVAL),
])
def test_experts_reject(lib, kw, status):
    assert moe(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(block=32), EUNSUPPORTED), (dict(rows=-1), EINVAL), (dict(cols=200), EINVAL), (dict(cols=0), EINVAL),
    (dict(cols=1 << 25), EUNSUPPORTED), (dict(rows=1 << 40), EUNSUPPORTED), (dict(grad=None), EINVAL), (dict(mask=None), EINVAL),
    (dict(out=None), EINVAL), (dict(grad=P[0] + 4), EALIGN), (dict(mask=P[1] + 8), EALIGN), (dict(out=P[2] + 2), EALIGN),
    (dict(out=P[0]), EINVAL), (dict(out=P[1] - 16), EINVAL), (dict(rows=0, grad=None, mask=None, out=None), OK),
])
def test_narrow_trust_backward_rejects(lib, kw, status):
    a = dict(dict(grad=P[0], mask=P[1], rows=4, cols=256, block=128, out=P[2]), **kw)
    assert lib.quest_trust_bwd_narrow(*a.values(), None) == status


def test_workspace_bytes(lib):
    f = lib.quest_moe_workspace_bytes
    # h and the products in fp32, h's codes; a slot (144 bytes) and three words for each row
    assert f(3, 8, 2048, 1024) == 24 * (4 * 2048 + 5 * 1024 + 156)
    assert f(64, 32, 32768, 8192) == 2048 * (4 * 32768 + 5 * 8192 + 156)
    for bad in ((-1, 2, 64, 64), (65, 2, 64, 64), (4, 0, 64, 64), (4, 33, 64, 64), (4, 2, 0, 64), (4, 2, 64, 0),
                (4, 2, 40000, 64), (4, 2, 64, 9000)):
        assert f(*bad) == 0


# ---------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("call,exc,msg", [
    (lambda: qa.quantize_fwd_i8(t(4), 128, 8), ValueError, "2-D"),
    (lambda: qa.quantize_fwd_i8(t(4, 256, dtype=torch.float16), 128, 8), TypeError, "float32 or bfloat16"),
    (lambda: qa.quantize_fwd_i8(t(4, 256), 128, 8, codes=t(4, 256)), TypeError, "codes must be"),
    (lambda: qa.quantize_fwd_i8(t(4, 256), 128, 8, codes=i8(4, 255)), ValueError, "codes must have shape"),
    (lambda: qa.quantize_fwd_i8(t(4, 256), 128, 8, scale=t(5)), ValueError, "scale must have shape"),
    (lambda: qa.quantize_fwd_i8(t(4, 256), 128, 8, mask=i8(4, 32)), TypeError, "mask must be"),
    (lambda: qa.quantize_fwd_i8(t(4, 256), 128, 8), ValueError, "GPU tensor"),
    (lambda: qa.dequantize_i8(i8(256), t(4), 8), ValueError, "2-D"),
    (lambda: qa.dequantize_i8(t(4, 256), t(4), 8), TypeError, "codes must be"),
    (lambda: qa.dequantize_i8(i8(4, 256), t(3), 8), ValueError, "scale must have shape"),
    (lambda: qa.dequantize_i8(i8(4, 256), t(4), 8, out=t(4, 255)), ValueError, "out must have shape"),
    (lambda: qa.dequantize_i8(i8(4, 256), t(4), 8, out_dtype=torch.float16), TypeError, "float32 or bfloat16"),
    (lambda: qa.trust_bwd_narrow(t(256), t(32, dtype=torch.uint8), 128), ValueError, "2-D"),
    (lambda: qa.trust_bwd_narrow(t(4, 256, dtype=torch.bfloat16), t(128, dtype=torch.uint8), 128), TypeError, "grad must be"),
    (lambda: qa.trust_bwd_narrow(t(4, 256), t(127, dtype=torch.uint8), 128), ValueError, "mask"),
    (lambda: qa.trust_bwd_narrow(t(4, 256), t(128, dtype=torch.uint8), 128, out=t(4, 256)), TypeError, "out must be"),
    (lambda: qa.trust_bwd_narrow(t(4, 256), t(128, dtype=torch.uint8), 128), ValueError, "GPU tensor"),
    (lambda: qa.gemm_i8(i8(256), t(4), 8, i8(5, 256), t(5), 8), ValueError, "a must be a 2-D"),
    (lambda: qa.gemm_i8(i8(4, 256), t(4), 8, i8(5), t(5), 8), ValueError, "b must be a 2-D"),
    (lambda: qa.gemm_i8(t(4, 256), t(4), 8, i8(5, 256), t(5), 8), TypeError, "a must be"),
    (lambda: qa.gemm_i8(i8(4, 256), t(4), 8, t(5, 256, dtype=torch.uint8), t(5), 8), TypeError, "b must be"),
    (lambda: qa.gemm_i8(i8(4, 256), t(4), 8, i8(5, 192), t(5), 8), ValueError, "b must have shape"),
    (lambda: qa.gemm_i8(i8(4, 256), t(5), 8, i8(5, 256), t(5), 8), ValueError, "a_scale must have shape"),
    (lambda: qa.gemm_i8(i8(4, 256), t(4), 8, i8(5, 256), t(5, dtype=torch.float64), 8), TypeError, "b_scale must be"),
    (lambda: qa.gemm_i8(i8(4, 256), t(4), 8, i8(5, 256), t(5), 8, out=t(5, 4)), ValueError, "out must have shape"),
    (lambda: qa.gemm_i8(i8(4, 256), t(4), 8, i8(5, 256), t(5), 8, out_dtype=torch.float64), TypeError, "float32 or bfloat16"),
    (lambda: qa.gemm_i8(i8(4, 256), t(4), 8, i8(5, 256), t(5), 8), ValueError, "GPU tensor"),
])
def test_binding_rejects(lib, call, exc, msg):
    with pytest.raises(exc, match=msg):
        call()


def experts_args(n=3, e=8, k=256, m=128, **kw):
    return dict(dict(x=i8(n, k), x_scale=t(n), x_bits=8, logits=t(n, e), gate=i8(e, m, k), gate_scale=t(e, m), up=i8(e, m, k),
                     up_scale=t(e, m), down=i8(e, k, m), down_scale=t(e, k), w_bits=8, top_k=2), **kw)


@pytest.mark.parametrize("kw,exc,msg", [
    (dict(x=i8(256)), ValueError, "x must be a 2-D"), (dict(x=t(3, 256)), TypeError, "x must be"),
    (dict(x_scale=t(4)), ValueError, "x_scale must have shape"), (dict(logits=t(8)), ValueError, "2-D"),
    (dict(logits=t(4, 8)), ValueError, "logits must have shape"), (dict(logits=t(3, 8, dtype=torch.float16)), TypeError, "float32"),
    (dict(gate=i8(8, 128)), ValueError, "3-D"), (dict(gate=t(8, 128, 256)), ValueError, "3-D"),
    (dict(gate=i8(7, 128, 256)), ValueError, "gate must have shape"), (dict(up=i8(8, 128, 255)), ValueError, "up must have shape"),
    (dict(up=t(8, 128, 256, dtype=torch.uint8)), TypeError, "up must be"), (dict(down=i8(8, 128, 256)), ValueError, "down must have"),
    (dict(gate_scale=t(8, 127)), ValueError, "gate_scale must have"), (dict(down_scale=t(8, 128)), ValueError, "down_scale must"),
    (dict(gate=t(8, 128, 128, dtype=torch.uint8)), ValueError, "packed codes"), (dict(top_k=0), ValueError, "top_k is 1"),
    (dict(top_k=9), ValueError, "top_k is 1"), (dict(act="relu"), ValueError, "act must be one of"),
    (dict(out=t(3, 255)), ValueError, "out must have shape"), (dict(out_dtype=torch.float16), TypeError, "float32 or bfloat16"),
    (dict(), ValueError, "GPU tensor"),
])
def test_experts_binding_rejects(lib, kw, exc, msg):
    with pytest.raises(exc, match=msg):
        qa.moe_fwd(**experts_args(**kw))


# ---------------------------------------------------------------------------
# The modules
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kw", [dict(grid="fp4"), dict(grid="sparse24"), dict(bits_x=9), dict(bits_w=0)])
def test_linear_rejects(kw):
    with pytest.raises(ValueError, match="8-bit integers"):
        QuestLinear(256, 64, int8=True, **kw)
    with pytest.raises(ValueError, match="8-bit integers"):
        quest_linear(t(2, 256), t(4, 256), int8=True, **kw)


def test_linear_too_wide():
    with pytest.raises(ValueError, match="8-bit integers"):
        QuestLinear(32768 + 128, 8, int8=True)


def test_linear_on_the_cpu_refuses(lib):
    layer = QuestLinear(256, 64, bits_x=8, bits_w=8, int8=True)
    for call in (lambda: layer(t(3, 256)), layer.freeze):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


@pytest.mark.parametrize("kw,exc", [
    (dict(features=200), ValueError), (dict(width=192), ValueError), (dict(block=96), ValueError), (dict(bits_x=0), ValueError),
    (dict(bits_w=9), ValueError), (dict(bits_h=9), ValueError), (dict(width=8320), ValueError), (dict(experts=257), ValueError),
    (dict(top_k=0), ValueError), (dict(top_k=9), ValueError), (dict(act="relu"), ValueError), (dict(experts=0), ValueError),
    (dict(compute_dtype=torch.float16), TypeError),
])
def test_experts_module_rejects(kw, exc):
    with pytest.raises(exc):
        QuestMoE(**dict(dict(features=256, width=256, experts=8, top_k=2), **kw))


def test_experts_on_the_cpu_refuse(lib):
    layer = QuestMoE(128, 128, 4, 2)
    assert [n for n, _ in layer.named_parameters()] == ["router", "gate_up", "down"]
    with pytest.raises(ValueError, match="GPU tensor"):
        layer(t(3, 128))
    with pytest.raises(ValueError, match="the last axis of x has 100"):
        layer(t(3, 100))


@pytest.mark.parametrize("over_all", [False, True])
def test_route_follows_the_definition(over_all):
    """Ranks with ties and masks as the oracle's, weights as the softmax over the chosen or all."""
    g = torch.Generator().manual_seed(1)
    logits = torch.randint(0, 4, (20, 12), generator=g).float()
    logits[3, 4:] = -float("inf")
    weight, index = route(logits, 4, over_all)
    for i, experts in enumerate(mo.chosen(logits.double().numpy(), 4)):
        assert index[i, :len(experts)].tolist() == experts
        e = np.exp(logits[i].double().numpy())
        want = e[experts] / (e.sum() if over_all else e[experts].sum())
        # exponentials, their sum of at most 12 and the quotient
        assert (np.abs(weight[i, :len(experts)].double().numpy() - want) <= 20 * mo.U * want).all()


def test_oracle_of_one_token():
    """The oracle's layer by hand: one expert of two columns' worth of blocks, no rounding in the way."""
    x, w = np.ones((1, 64)), np.eye(64)[None]
    y, _ = mo.moe(x, np.zeros((1, 1)), w, w, w, 1, 64, 8, "silu", False)
    # h is constant, so one transformed entry holds it all: the outermost level, (2^8 - 1) / 2 steps, in place 0
    h = 1 / (1 + np.exp(-1.0))
    from oracle import quest_oracle as qo

    s = qo.fit_alpha(8) * h
    want = np.full(64, s / 255)  # zeros take the level above
    want[0] = s
    assert np.allclose(y[0], want, rtol=1e-12)
