"""Argument checks of the layer norm, 8-bit checkpoint and gated product calls, on the CPU.

No call launches a kernel: the C entries get arguments that they must reject
before touching a buffer (the pointers are never dereferenced) or empty sizes,
and the binding gets CPU tensors, whose sizes and types it checks before their
device.
"""
from __future__ import annotations

import os
import re

import numpy as np
import pytest
import torch
from scipy.special import erfcx

import quantization_aware_amd as qa

OK, EINVAL, EUNSUPPORTED, EALIGN = qa.QUEST_OK, qa.QUEST_EINVAL, qa.QUEST_EUNSUPPORTED, qa.QUEST_EALIGN
P = [0x10000000 * (i + 1) for i in range(16)]  # aligned and far apart


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qa.LIB_PATH):
        pytest.fail("libquest.so is not built; run `python -m quantization_aware_amd.build`")
    return qa.load_library()


# ---------------------------------------------------------------------------
# The C entries
# ---------------------------------------------------------------------------

def save(lib, x=P[0], dt=qa.QUEST_BF16, rows=4, cols=100, codes=P[1], scale=P[2]):
    return lib.quest_act8_save(x, dt, rows, cols, codes, scale, None)


def load(lib, codes=P[0], scale=P[1], rows=4, cols=100, out=P[2], dt=qa.QUEST_BF16):
    return lib.quest_act8_load(codes, scale, rows, cols, out, dt, None)


def norm(lib, x=P[0], dt=qa.QUEST_BF16, rows=4, cols=100, w=P[1], b=P[2], pdt=qa.QUEST_F32, eps=1e-5, y=P[3],
         mean=P[4], rstd=P[5], codes=None, scale=None):
    return lib.quest_layer_norm_fwd(x, dt, rows, cols, w, b, pdt, eps, y, mean, rstd, codes, scale, None)


def norm_bwd(lib, dy=P[0], dt=qa.QUEST_BF16, rows=4, cols=100, x=P[1], mean=P[2], codes=None, scale=None, rstd=P[3],
             w=P[4], pdt=qa.QUEST_F32, dx=P[5], dw=P[6], db=P[7], ws=P[8]):
    return lib.quest_layer_norm_bwd(dy, dt, rows, cols, x, mean, codes, scale, rstd, w, pdt, dx, dw, db, ws, None)


def gated(lib, x=P[0], xs=P[1], n=4, xb=4, g=P[2], gs=P[3], u=P[4], us=P[5], m=100, wb=4, k=256, act=0, out=P[6],
          dt=qa.QUEST_BF16, gc=None, ge=None, uc=None, ue=None):
    return lib.quest_gated_fwd(x, xs, n, xb, g, gs, u, us, m, wb, k, act, out, dt, gc, ge, uc, ue, None)


def gated_bwd(lib, dh=P[0], dt=qa.QUEST_BF16, rows=4, cols=100, gc=P[1], ge=P[2], uc=P[3], ue=P[4], act=0, out=P[5]):
    return lib.quest_gated_bwd(dh, dt, rows, cols, gc, ge, uc, ue, act, out, None)


def test_empty_calls_are_noops(lib):
    assert save(lib, x=None, rows=0, codes=None, scale=None) == OK
    assert load(lib, codes=None, scale=None, rows=0, out=None) == OK
    assert norm(lib, x=None, rows=0, w=None, b=None, y=None, mean=None, rstd=None) == OK
    assert norm_bwd(lib, dy=None, rows=0, x=None, mean=None, rstd=None, w=None, dx=None, dw=None, db=None,
                    ws=None) == OK
    none = dict(x=None, xs=None, g=None, gs=None, u=None, us=None, out=None)
    assert gated(lib, n=0, **none) == OK and gated(lib, m=0, **none) == OK
    bnone = dict(dh=None, gc=None, ge=None, uc=None, ue=None, out=None)
    assert gated_bwd(lib, rows=0, **bnone) == OK and gated_bwd(lib, cols=0, **bnone) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL), (dict(cols=(1 << 20) + 1), EUNSUPPORTED),
    (dict(rows=1 << 40, cols=1024), EUNSUPPORTED), (dict(x=None), EINVAL), (dict(codes=None), EINVAL),
    (dict(scale=None), EINVAL), (dict(x=P[0] + 8), EALIGN), (dict(codes=P[1] + 4), EALIGN),
    (dict(scale=P[2] + 1), EALIGN), (dict(codes=P[0] + 16), EINVAL), (dict(scale=P[1] + 384), EINVAL),
    (dict(scale=P[0]), EINVAL),
])
def test_act8_save_rejects(lib, kw, status):
    assert save(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=-1), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=-3), EINVAL), (dict(cols=(1 << 20) + 1), EUNSUPPORTED),
    (dict(out=None), EINVAL), (dict(codes=None), EINVAL), (dict(scale=None), EINVAL), (dict(out=P[2] + 2), EALIGN),
    (dict(out=P[0] + 16), EINVAL), (dict(out=P[1]), EINVAL),
])
def test_act8_load_rejects(lib, kw, status):
    assert load(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), EINVAL), (dict(pdt=2), EINVAL), (dict(eps=0.0), EINVAL), (dict(eps=-1e-5), EINVAL),
    (dict(eps=1e-60), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(eps=1e39), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL), (dict(cols=32769), EUNSUPPORTED),
    (dict(rows=1 << 50), EUNSUPPORTED), (dict(x=None), EINVAL), (dict(y=None), EINVAL), (dict(codes=P[6]), EINVAL),
    (dict(scale=P[6]), EINVAL), (dict(y=P[0]), EINVAL), (dict(y=P[1]), EINVAL), (dict(mean=P[5]), EINVAL),
    (dict(codes=P[6], scale=P[3] + 16), EINVAL), (dict(w=P[1] + 2), EALIGN), (dict(b=P[2] + 4), EALIGN),
    (dict(mean=P[4] + 4), EALIGN), (dict(rstd=P[5] + 8), EALIGN), (dict(codes=P[6] + 1, scale=P[7]), EALIGN),
])
def test_layer_norm_fwd_rejects(lib, kw, status):
    assert norm(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=9), EINVAL), (dict(pdt=9), EINVAL), (dict(rows=-2), EINVAL), (dict(cols=0), EINVAL),
    (dict(cols=40000), EUNSUPPORTED), (dict(dy=None), EINVAL), (dict(rstd=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(dx=None, dw=None, db=None), EINVAL), (dict(x=None), EINVAL), (dict(mean=None), EINVAL),
    (dict(codes=P[9]), EINVAL), (dict(scale=P[9]), EINVAL), (dict(codes=P[9], scale=P[10]), EINVAL),
    (dict(x=None, mean=None), EINVAL), (dict(x=None, mean=None, codes=P[9]), EINVAL),
    (dict(dx=P[0]), EINVAL), (dict(dx=P[1]), EINVAL), (dict(dw=P[4]), EINVAL), (dict(db=P[6]), EINVAL),
    (dict(ws=P[5]), EINVAL), (dict(ws=P[8] + 4), EALIGN), (dict(dw=P[6] + 8), EALIGN), (dict(dx=P[5] + 2), EALIGN),
])
def test_layer_norm_bwd_rejects(lib, kw, status):
    assert norm_bwd(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(xb=0), EUNSUPPORTED), (dict(xb=5), EUNSUPPORTED), (dict(wb=8), EUNSUPPORTED), (dict(dt=3), EINVAL),
    (dict(act=2), EINVAL), (dict(act=-1), EINVAL), (dict(n=-1), EINVAL), (dict(m=-1), EINVAL), (dict(k=0), EINVAL),
    (dict(k=200), EUNSUPPORTED), (dict(k=65536 + 128), EUNSUPPORTED), (dict(m=(1 << 20) + 1), EUNSUPPORTED),
    (dict(n=(1 << 30) + 1), EUNSUPPORTED), (dict(n=1 << 30, m=1 << 20), EUNSUPPORTED), (dict(x=None), EINVAL),
    (dict(xs=None), EINVAL), (dict(g=None), EINVAL), (dict(gs=None), EINVAL), (dict(u=None), EINVAL),
    (dict(us=None), EINVAL), (dict(out=None), EINVAL), (dict(gc=P[7]), EINVAL), (dict(gc=P[7], ge=P[8]), EINVAL),
    (dict(gc=P[7], ge=P[8], uc=P[9]), EINVAL), (dict(ue=P[9]), EINVAL), (dict(out=P[0]), EINVAL),
    (dict(out=P[5]), EINVAL), (dict(gc=P[7], ge=P[8], uc=P[7], ue=P[10]), EINVAL),
    (dict(gc=P[7], ge=P[8], uc=P[9], ue=P[6]), EINVAL), (dict(out=P[6] + 8), EALIGN), (dict(gs=P[3] + 4), EALIGN),
    (dict(gc=P[7], ge=P[8] + 1, uc=P[9], ue=P[10]), EALIGN),
])
def test_gated_fwd_rejects(lib, kw, status):
    assert gated(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), EINVAL), (dict(act=2), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL),
    (dict(cols=(1 << 20) + 1), EUNSUPPORTED), (dict(rows=1 << 30, cols=1 << 20), EUNSUPPORTED), (dict(dh=None), EINVAL),
    (dict(gc=None), EINVAL), (dict(ge=None), EINVAL), (dict(uc=None), EINVAL), (dict(ue=None), EINVAL),
    (dict(out=None), EINVAL), (dict(out=P[0]), EINVAL), (dict(out=P[1]), EINVAL), (dict(out=P[5] + 2), EALIGN),
])
def test_gated_bwd_rejects(lib, kw, status):
    assert gated_bwd(lib, **kw) == status


def test_sizes(lib):
    assert lib.quest_act8_scale_bytes(3, 1) == 3 and lib.quest_act8_scale_bytes(3, 33) == 6
    assert lib.quest_act8_scale_bytes(-1, 33) == 0 and lib.quest_act8_scale_bytes(2, 0) == 0
    assert lib.quest_layer_norm_workspace_bytes(0, 64) == 0
    assert lib.quest_layer_norm_workspace_bytes(5, 40000) == 0
    assert lib.quest_layer_norm_workspace_bytes(1, 64) == 2 * 64 * 4
    # bounded by the workgroups that walk the rows
    assert lib.quest_layer_norm_workspace_bytes(1 << 20, 2048) == lib.quest_layer_norm_workspace_bytes(1 << 21, 2048)


# ---------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------

def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def pair(rows, cols):
    return t(rows, cols, dtype=torch.int8), t(rows, -(-cols // 32), dtype=torch.uint8)


def test_well_formed_cpu_tensors_reach_the_device_check(lib):
    for call in (lambda: qa.act8_save(t(4, 40)), lambda: qa.act8_load(*pair(4, 40)),
                 lambda: qa.layer_norm_fwd(t(4, 40), t(40), t(40)),
                 lambda: qa.layer_norm_bwd(t(4, 40), t(4), t(40), x=t(4, 40), mean=t(4)),
                 lambda: qa.layer_norm_bwd(t(4, 40), t(4), t(40), act8=pair(4, 40)),
                 lambda: qa.gated_fwd(**gated_args()),
                 lambda: qa.gated_bwd(t(4, 40), pair(4, 40), pair(4, 40))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


@pytest.mark.parametrize("call,exc,msg", [
    (lambda: qa.act8_save(t(40)), ValueError, "2-D"),
    (lambda: qa.act8_save(t(4, 40, dtype=torch.float16)), TypeError, "float32 or bfloat16"),
    (lambda: qa.act8_save(t(4, 40), codes=t(4, 39, dtype=torch.int8)), ValueError, "codes must have shape"),
    (lambda: qa.act8_save(t(4, 40), codes=t(4, 40, dtype=torch.uint8)), TypeError, "codes must be"),
    (lambda: qa.act8_save(t(4, 40), scale=t(4, 1, dtype=torch.uint8)), ValueError, "scale must have shape"),
    (lambda: qa.act8_load(t(4, 40, dtype=torch.int8), t(4, 3, dtype=torch.uint8)), ValueError, "scale must have shape"),
    (lambda: qa.act8_load(*pair(4, 40), out=t(4, 41)), ValueError, "out must have shape"),
    (lambda: qa.act8_load(*pair(4, 40), out=t(4, 40, dtype=torch.float16)), TypeError, "float32 or bfloat16"),
    (lambda: qa.layer_norm_fwd(t(4, 40), t(41)), ValueError, "weight must have shape"),
    (lambda: qa.layer_norm_fwd(t(4, 40), t(40), t(40, dtype=torch.bfloat16)), TypeError, "share one type"),
    (lambda: qa.layer_norm_fwd(t(4, 40), t(40, dtype=torch.float64)), TypeError, "float32 or bfloat16"),
    (lambda: qa.layer_norm_fwd(t(4, 40), out=t(4, 40, dtype=torch.bfloat16)), TypeError, "out must be"),
    (lambda: qa.layer_norm_bwd(t(4, 40), t(4), t(40)), ValueError, "give x and mean, or act8"),
    (lambda: qa.layer_norm_bwd(t(4, 40), t(4), t(40), x=t(4, 40)), ValueError, "give x and mean, or act8"),
    (lambda: qa.layer_norm_bwd(t(4, 40), t(4), t(40), x=t(4, 40), mean=t(4), act8=pair(4, 40)), ValueError, "or act8"),
    (lambda: qa.layer_norm_bwd(t(4, 40), t(4), act8=pair(4, 40), input_grad=False), ValueError, "no gradient"),
    (lambda: qa.layer_norm_bwd(t(4, 40), t(5), t(40), act8=pair(4, 40)), ValueError, "rstd must have shape"),
    (lambda: qa.layer_norm_bwd(t(4, 40), t(4), t(40), x=t(4, 40, dtype=torch.bfloat16), mean=t(4)), TypeError, "x must"),
    (lambda: qa.layer_norm_bwd(t(4, 40), t(4), t(40), act8=pair(3, 40)), ValueError, "act8 codes must have shape"),
    (lambda: qa.layer_norm_bwd(t(4, 40), t(4), t(40), act8=t(4, 40)), TypeError, "pair"),
    (lambda: qa.layer_norm_bwd(t(4, 40), t(4), act8=pair(4, 40), bias_grad=True, param_dtype=torch.float16), TypeError,
     "parameter gradients"),
    (lambda: qa.gated_bwd(t(4, 40), pair(4, 40), pair(4, 41)), ValueError, "up8 codes must have shape"),
    (lambda: qa.gated_bwd(t(4, 40), pair(4, 40), pair(4, 40), act="relu"), ValueError, "act must be one of"),
    (lambda: qa.gated_bwd(t(4, 40), pair(4, 40), pair(4, 40), out=t(4, 40)), ValueError, "out must have shape"),
])
def test_binding_rejects(lib, call, exc, msg):
    with pytest.raises(exc, match=msg):
        call()


def gated_args(n=40, m=24, k=256, **kw):
    u8 = lambda rows: torch.zeros(qa.operand_bytes(rows, k), dtype=torch.uint8)
    return dict(dict(x=u8(n), x_scale=t(n), n=n, x_bits=4, gate=u8(m), gate_scale=t(m), up=u8(m), up_scale=t(m), m=m,
                     w_bits=4, k=k), **kw)


@pytest.mark.parametrize("kw,exc,msg", [
    (dict(x=torch.zeros(1, dtype=torch.uint8)), ValueError, "x too small"),
    (dict(gate=torch.zeros(1, dtype=torch.uint8)), ValueError, "gate too small"),
    (dict(up=torch.zeros(1, dtype=torch.uint8)), ValueError, "up too small"),
    (dict(up=torch.zeros(1 << 16, dtype=torch.int8)), TypeError, "up must be"),
    (dict(x_scale=torch.zeros(39)), ValueError, "x_scale too small"),
    (dict(gate_scale=torch.zeros(23)), ValueError, "gate_scale too small"),
    (dict(up_scale=torch.zeros(24, dtype=torch.float64)), TypeError, "up_scale must be"),
    (dict(act="relu"), ValueError, "act must be one of"),
    (dict(out_dtype=torch.float16), TypeError, "float32 or bfloat16"),
    (dict(out=torch.zeros(40, 25)), ValueError, "out must have shape"),
])
def test_gated_fwd_binding_rejects(lib, kw, exc, msg):
    with pytest.raises(exc, match=msg):
        qa.gated_fwd(**gated_args(**kw))


def test_non_contiguous_tensors_are_refused(lib):
    # contiguity and device are one check of the binding, which CPU tensors do not pass
    for call in (lambda: qa.act8_save(t(40, 4).t()), lambda: qa.layer_norm_fwd(t(4, 80)[:, ::2])):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------------------
# The modules
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kw,exc", [
    (dict(features=192, width=256), ValueError), (dict(features=256, width=256, block=96), ValueError),
    (dict(features=256, width=200), ValueError), (dict(features=256, width=256, bits_x=5), ValueError),
    (dict(features=256, width=256, bits_w=0), ValueError), (dict(features=256, width=256, act="relu"), ValueError),
    (dict(features=256, width=256, compute_dtype=torch.float16), TypeError),
])
def test_block_rejects(kw, exc):
    from quantization_aware_amd.feedforward import QuestFeedForward

    with pytest.raises(exc):
        QuestFeedForward(**kw)


def test_modules_on_the_cpu_refuse(lib):
    from quantization_aware_amd.feedforward import LayerNorm, QuestFeedForward, layer_norm, quest_gated

    ff = QuestFeedForward(128, 256)
    assert [n for n, _ in ff.named_parameters()] == ["gate", "up", "norm.weight", "norm.bias", "down.weight"]
    with pytest.raises(ValueError, match="GPU tensor"):
        ff(t(3, 128))
    with pytest.raises(ValueError, match="GPU tensor"):
        layer_norm(t(3, 128))
    with pytest.raises(ValueError, match="the last axis of x has 100"):
        LayerNorm(128)(t(3, 100))
    with pytest.raises(ValueError, match="got"):
        quest_gated(t(3, 128), t(8, 256), t(8, 256))


def test_frozen_block_keeps_nothing_for_a_backward_pass(monkeypatch):
    """Frozen forwards carry no gradient, so their norm writes no checkpoint, also where gradients are enabled."""
    from quantization_aware_amd import feedforward as ff_mod

    asked = []

    def norm_fwd(x, weight, bias, eps, act8=False):
        asked.append(act8)
        return x + weight + bias, t(x.shape[0]), t(x.shape[0]), pair(*x.shape) if act8 else None

    monkeypatch.setattr(ff_mod, "layer_norm_fwd", norm_fwd)
    monkeypatch.setattr(ff_mod, "quantize_fwd_op", lambda x, *a, **kw: (None, None, None, x))
    monkeypatch.setattr(ff_mod, "gated_fwd", lambda x, *a, **kw: (x.repeat(1, 2), None, None))
    ff = ff_mod.QuestFeedForward(128, 256)
    ff.down.forward = lambda h: h[..., :128]
    ff._frozen = [(None, None), (None, None)]
    ff.eval()
    x = t(3, 5, 128).requires_grad_()
    y = ff(x)
    assert asked == [False]
    assert y.shape == (3, 5, 128) and not y.requires_grad


def test_gelu_fit():
    """normal_cdf's coefficients are the halved minimax fit of erfc(z) exp(z^2) by a polynomial of degree 8 in
    t = 1 / (1 + 0.325 z), in relative error over 0 <= z <= 9.4: found here by exchange of its extrema in 64 bits,
    and rounded to fp32."""
    p, deg = 0.325, 8
    src = open(os.path.join(os.path.dirname(qa.__file__), "csrc", "quest_gated.hip")).read()
    body = src[src.index("float normal_cdf("):]
    body = body[:body.index("const float q =")]
    held = [float(a or b) for a, b in re.findall(r"float p = ([-0-9.e]+)f;|fmaf\(p, t, ([-0-9.e]+)f\)", body)]
    scale = float(re.search(r"fmaf\(fabsf\(g\), ([0-9.]+)f, 1\.0f\)", body).group(1))
    assert len(held) == deg + 1 and abs(scale - p / 2 ** 0.5) <= 2.0 ** -24 * scale * 2

    def f(t):
        return erfcx((1 / t - 1) / p)

    lo = 1 / (1 + p * 9.4)
    grid = np.linspace(lo, 1.0, 100001)
    want = f(grid)
    x = (lo + 1) / 2 + (1 - lo) / 2 * np.cos(np.pi * np.arange(deg + 1, -1, -1) / (deg + 1))
    for _ in range(30):
        rows = np.hstack([np.vander(x, deg + 1) / f(x)[:, None], ((-1.0) ** np.arange(deg + 2))[:, None]])
        c = np.linalg.solve(rows, np.ones(deg + 2))[:-1]
        r = np.polyval(c, grid) / want - 1
        edges = np.flatnonzero(np.diff(np.sign(r))) + 1
        ext = [s + np.argmax(np.abs(r[s:e])) for s, e in zip([0, *edges], [*edges, len(grid)])]
        assert len(ext) == deg + 2
        x = grid[ext]
    top = np.abs(r).max()
    assert 4.4e-8 < top < 4.6e-8 and np.abs(r[ext]).min() > 0.999 * top  # levelled: the best there is
    assert (np.float32(held) == np.float32(c / 2)).all()
