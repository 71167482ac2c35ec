"""Host-side logic of the linear layer in 8-bit integers (no GPU)."""
from __future__ import annotations

import pytest
import torch

from quantization_aware_amd.linear import QuestLinear, quest_linear_int8


@pytest.mark.parametrize("dtype", [torch.int32, torch.bool, None, "bf16"])
def test_frozen_product_refuses_other_types(dtype):
    codes, scale = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)
    with pytest.raises(TypeError, match="floating-point"):
        quest_linear_int8(torch.zeros(2, 64), codes, scale, 8, block=64, out_dtype=dtype)


def test_a_module_from_before_int8_is_the_default_layer():
    """A whole QuestLinear that was pickled before it had int8 lacks the attribute."""
    layer = QuestLinear(256, 64, bits_x=8, bits_w=8)
    del layer.__dict__["int8"]
    layer.to(torch.float32).load_state_dict(layer.state_dict())
    assert layer.int8 is False
    with pytest.raises(ValueError, match="FP6"):
        layer.freeze()
