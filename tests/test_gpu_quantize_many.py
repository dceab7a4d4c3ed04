"""``quantize_fp8`` of so many blocks that a warp has several at a time, against its definition in 64 bits."""
import pytest
import torch

import prompt_util as P

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# 155648 blocks on 152 SMs are where the other kernel begins; the last blocks of a row are short, and the last four not all there
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,k", [(17293, 1040), (17295, 1040), (155647, 128), (155649, 48), (25943, 784)])
def test_many_blocks(m, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(m)
    x = (torch.randn((m, k), generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (m, 1), generator=g, device="cuda").float())).to(dtype)
    x[5, :16] = 0.0
    room = torch.zeros((m + 2, k), device="cuda").to(E4M3)
    codes, scales = mk.quantize_fp8(x, codes=room[1:m + 1])
    want, s = P.quantized(x)                                # (64 bits, on the device)
    assert torch.equal(scales.double(), s) and torch.equal(codes.double(), want)
    assert not room.view(torch.uint8)[0].any() and not room.view(torch.uint8)[m + 1].any()
