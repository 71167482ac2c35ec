"""Host-side logic of the layer of experts (no GPU): what its backward pass allocates."""
from __future__ import annotations

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from quantization_aware_amd import experts
from quantization_aware_amd.experts import QuestMoE


@pytest.fixture
def plain_products(monkeypatch):
    """QuestMoE on ordinary products, without the library."""
    monkeypatch.setattr(experts, "quest_linear",
                        lambda x, w, **kw: torch.nn.functional.linear(x.float(), w.float()).to(kw["compute_dtype"]))


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
