"""The dequantiser of codes one a byte on tensors whose offsets pass 32 bits in each of the kernel's counts."""
from __future__ import annotations

import pytest
import torch

import quantization_aware_amd as qa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,dtype", [(2 ** 19 + 40, 32768, torch.float32), (1_100_000, 32704, torch.bfloat16)])
def test_values_past_2_to_the_34_entries(rows, cols, dtype):
    """Outputs of 64 GiB and more: every sampled row is the one a call of that row alone gives, the first ones too,
    and the rows behind the last are left as they were.  (fp32: 2^34 entries, 2^32 pieces of 16 bytes; bf16: 2^35.)"""
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qa.load_library()
    dev = torch.device("cuda", 0)
    print(f"[gpu-i8-large] {rows}x{cols} {dtype}", flush=True)
    torch.cuda.empty_cache()
    codes = torch.zeros((rows, cols), dtype=torch.int8, device=dev)
    per_launch = 2 ** 30 // (cols // 16)
    at = torch.tensor(sorted({0, 1, 39, per_launch - 1, per_launch, per_launch + 1, rows // 2, rows - 2, rows - 1}), device=dev)
    at = torch.unique(torch.cat([at, torch.arange(0, rows, 4999, device=dev)]))
    codes[at] = torch.randint(-128, 128, (len(at), cols), dtype=torch.int8, device=dev)
    scale = torch.rand(rows, device=dev) + 0.5
    buf = torch.full((rows + 3, cols), 7.0, dtype=dtype, device=dev)
    qa.dequantize_i8(codes, scale, 8, out=buf[:rows])
    want = qa.dequantize_i8(codes[at], scale[at], 8, out_dtype=dtype)
    assert torch.equal(buf[at], want) and (buf[rows:] == 7.0).all()
    # (rows of zeros between them: scale / 255 each)
    other = at[:-1] + 2500
    other = other[other < rows]
    other = other[~torch.isin(other, at)]
    assert torch.equal(buf[other], qa.dequantize_i8(codes[other], scale[other], 8, out_dtype=dtype))
    del codes, buf
    torch.cuda.empty_cache()
