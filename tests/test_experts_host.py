"""Host-side logic of the layer of experts (no GPU): the choice of experts, and what its backward pass allocates."""
from __future__ import annotations

import math

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from quantization_aware_amd import experts
from quantization_aware_amd.experts import QuestMoE, route

INF = math.inf


@pytest.fixture
def plain_products(monkeypatch):
    """QuestMoE on ordinary products, without the library."""
    monkeypatch.setattr(experts, "quest_linear",
                        lambda x, w, **kw: torch.nn.functional.linear(x.float(), w.float()).to(kw["compute_dtype"]))


@pytest.mark.parametrize("over_all", [False, True])
def test_route_without_experts_to_take(over_all):
    logits = torch.tensor([[-INF, -INF, -INF], [1.0, -INF, 2.0], [-INF, 0.5, -INF], [math.nan, 0.0, 0.0],
                           [INF, 0.0, 0.0]], requires_grad=True)
    weight, index = route(logits, 2, over_all)
    assert torch.equal(weight[0], torch.zeros(2))
    a = 1 / (1 + math.exp(-1.0))
    assert torch.allclose(weight[1], torch.tensor([a, 1 - a])) and index[1].tolist() == [2, 0]
    assert weight[2].tolist() == [1.0, 0.0] and index[2, 0] == 1
    assert weight[3:].isnan().any(1).all()
    weight[:3].square().sum().backward()
    assert logits.grad[:3].isfinite().all() and (logits.grad[0] == 0).all()


def test_a_token_without_experts_gives_zeros(plain_products):
    moe = QuestMoE(64, 64, 3, 2, block=64, compute_dtype=torch.float32)
    with torch.no_grad():
        moe.router.fill_(-1e30)
        moe.router[1] = 0.0
        moe.gate_up[2].fill_(math.nan)  # an expert that is never taken
    x = torch.zeros(2, 64)
    x[0, 0] = 1e10  # logits -inf, 0, -inf
    x.requires_grad_()
    y = moe(x[:1])
    want = moe._linear(torch.nn.functional.silu(moe._linear(x[:1], moe.gate_up[1, :64], 4))
                       * moe._linear(x[:1], moe.gate_up[1, 64:], 4), moe.down[1], 4)
    assert torch.allclose(y, want) and y.isfinite().all()
    with torch.no_grad():
        moe.router.fill_(-1e30)
    y = moe(x[:1])
    y.sum().backward()
    assert (y == 0).all() and (x.grad == 0).all() and (moe.router.grad == 0).all()


def test_no_tokens_have_a_backward_pass(plain_products):
    moe = QuestMoE(64, 64, 3, 2, block=64)
    x = torch.zeros(0, 64, requires_grad=True)
    y = moe(x)
    assert y.shape == (0, 64) and y.dtype == torch.bfloat16
    y.sum().backward()
    assert x.grad.shape == (0, 64) and (moe.router.grad == 0).all()


def test_gradients_take_memory_in_proportion_to_the_weights(plain_products):
    """The backward pass makes each weight's whole gradient once, however many experts there are."""
    e = 16
    moe = QuestMoE(64, 64, e, 2, block=64, compute_dtype=torch.float32)
    made = {tuple(moe.gate_up.shape): 0, tuple(moe.down.shape): 0}

    class Count(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if isinstance(out, torch.Tensor) and tuple(out.shape) in made:
                made[tuple(out.shape)] += 1
            return out

    y = moe(torch.randn(40, 64))
    with Count():
        y.square().sum().backward()
    assert moe.gate_up.grad.shape == moe.gate_up.shape and moe.gate_up.grad.abs().sum() > 0
    # (the gradient, and its detached alias as autograd keeps it)
    assert all(count <= 3 for count in made.values()), made


@pytest.mark.parametrize("grad", [True, False])
def test_a_token_of_nan_keeps_to_itself(plain_products, grad):
    moe = QuestMoE(64, 64, 3, 2, block=64, compute_dtype=torch.float32)
    x = torch.randn(4, 64)
    x[2, 5] = math.nan
    with torch.set_grad_enabled(grad):
        y = moe(x)
    assert y[2].isnan().all() and y[[0, 1, 3]].isfinite().all()
