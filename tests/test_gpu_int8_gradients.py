"""Gradients of the quantised layers: whose memory they hold."""
from __future__ import annotations

import pytest
import torch

import quantization_aware_amd as qa
from quantization_aware_amd.linear import quest_linear

pytestmark = pytest.mark.gpu


def log(msg: str) -> None:
    print(f"[gpu-int8-gradients] {msg}", flush=True)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    return torch.device("cuda", 0)


TYPES = [(torch.bfloat16, torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32, torch.bfloat16),
         (torch.float32, torch.bfloat16, torch.float32), (torch.float32, torch.float32, torch.float32)]


def owns(grad):
    return grad.untyped_storage().nbytes() == grad.numel() * grad.element_size()


@pytest.mark.parametrize("x_dtype,w_dtype,compute", TYPES)
@pytest.mark.parametrize("n,bits_x,bits_w", [(64, 8, 8), (64, 4, 4), (63, 8, 8), (64, 8, 6)])
def test_gradients_hold_their_own_memory(dev, x_dtype, w_dtype, compute, n, bits_x, bits_w):
    """weight.grad outlives the step: it keeps nothing alive but itself, however x's and w's codes are laid out."""
    log(f"memory of gradients n={n} {bits_x} and {bits_w} bits {x_dtype} {w_dtype} {compute}")
    x = torch.randn(n, 256, device=dev).to(x_dtype).requires_grad_()
    w = torch.randn(24, 256, device=dev).to(w_dtype).requires_grad_()
    quest_linear(x, w, bits_x=bits_x, bits_w=bits_w, compute_dtype=compute, int8=True).float().sum().backward()
    for t in (x, w):
        assert t.grad.dtype == t.dtype and t.grad.shape == t.shape and owns(t.grad)


@pytest.mark.parametrize("x_dtype,w_dtype,compute", TYPES)
@pytest.mark.parametrize("n", [64, 63])
def test_gradients_of_the_default_layer_hold_their_own_memory(dev, x_dtype, w_dtype, compute, n):
    """The same of the FP6 product's layer, whose codes are the rows of one tensor where n is a multiple of 4."""
    x = torch.randn(n, 256, device=dev).to(x_dtype).requires_grad_()
    w = torch.randn(24, 256, device=dev).to(w_dtype).requires_grad_()
    quest_linear(x, w, bits_x=4, bits_w=4, compute_dtype=compute).float().sum().backward()
    for t in (x, w):
        assert t.grad.dtype == t.dtype and t.grad.shape == t.shape and owns(t.grad)
