"""``quantize_q4`` of weights in any memory order (no GPU)."""
import pytest
import torch

import persistent_transformer_megakernel_gb300 as mk


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float64])
def test_strided_weights(zeros, dtype):
    w = torch.randn((256, 12), generator=torch.Generator().manual_seed(0)).to(dtype)
    wide = torch.zeros((12, 300), dtype=dtype)
    wide[:, 7:263] = w.t()
    for view in (w.t(), wide[:, 7:263], w.t()[::2]):
        for a, b in zip(mk.quantize_q4(view, 64, zeros), mk.quantize_q4(view.contiguous(), 64, zeros)):
            assert torch.equal(a, b) and a.is_contiguous()
