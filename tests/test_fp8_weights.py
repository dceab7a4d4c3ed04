"""``quantize_fp8_weight`` of weights that are no numbers (no GPU)."""
import math

import torch

import persistent_transformer_megakernel_gb300 as mk

E4M3 = torch.float8_e4m3fn


def test_nan_does_not_count_for_the_scale():
    w = torch.randn((200, 272), generator=torch.Generator().manual_seed(1)) * 0.02
    want, scales = mk.quantize_fp8_weight(w)
    bad = w.clone()
    at = (torch.tensor([0, 5, 130, 199]), torch.tensor([3, 140, 3, 271]))
    assert (bad[at].abs() < torch.tensor([448.0]) * scales[at[0] // 128, at[1] // 128]).all()   # (none is its block's largest)
    bad[at] = math.nan
    codes, s = mk.quantize_fp8_weight(bad)
    assert torch.equal(s, scales)
    assert torch.isnan(codes.float()[at]).all() and int(torch.isnan(codes.float()).sum()) == 4
    keep = ~torch.isnan(bad)
    assert torch.equal(codes.float()[keep], want.float()[keep])


def test_blocks_of_nothing_but_nan_and_zeros():
    w = torch.zeros((128, 256))
    w[3, :128] = math.nan
    codes, s = mk.quantize_fp8_weight(w)
    assert (s == 1).all() and torch.isnan(codes.float()[3, :128]).all() and int((codes.float() == 0).sum()) == 128 * 256 - 128
