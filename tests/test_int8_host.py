"""Host-side logic of the linear layer in 8-bit integers (no GPU)."""
from __future__ import annotations

import pytest
import torch

from quantization_aware_amd.linear import quest_linear_int8


@pytest.mark.parametrize("dtype", [torch.int32, torch.bool, None, "bf16"])
def test_frozen_product_refuses_other_types(dtype):
    codes, scale = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)
    with pytest.raises(TypeError, match="floating-point"):
        quest_linear_int8(torch.zeros(2, 64), codes, scale, 8, block=64, out_dtype=dtype)
