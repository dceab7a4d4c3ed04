"""The results that ``quantize_fp8`` makes: their sizes for the most rows, and memory of their own."""
import io

import pytest
import torch

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def test_the_most_rows():
    # 4 bytes a scale pass 2^31 here.  One row expanded, 8.6 GB of codes and 2.1 GB of scales; what is allocated behind the
    # call is not what it wrote
    m = 1 << 29
    row = torch.tensor([[1.0, -2.0, 448.0, 0.0, 3.0, -448.0, 7.0, 0.5] * 2], dtype=BF16, device="cuda")
    codes, scales = mk.quantize_fp8(row.expand(m, -1))
    more = torch.full((1 << 28,), 5.0, device="cuda")
    assert codes.shape == (m, 16) and scales.shape == (m, 1)
    assert codes.untyped_storage().nbytes() == 16 * m and scales.untyped_storage().nbytes() == 4 * m
    words = codes.view(torch.uint8).view(torch.int64)
    assert (words == words[0, 0]).all() and torch.equal(codes[m - 1].float(), row[0].float())
    assert (scales == 1).all() and (more == 5).all()


@pytest.mark.parametrize("m,k", [(0, 16), (1, 16), (5, 144), (300, 2048)])
def test_codes_and_scales_are_apart(m, k):
    codes, scales = mk.quantize_fp8(torch.ones((m, k), dtype=BF16, device="cuda"))
    assert codes.untyped_storage().nbytes() == m * k and scales.untyped_storage().nbytes() == 4 * m * -(-k // 128)
    want = scales.clone()
    codes.resize_(2 * m + 3, k).view(torch.uint8).fill_(255)
    assert torch.equal(scales, want)
    file = io.BytesIO()
    torch.save(scales, file)
    assert file.tell() < 4 * scales.numel() + 2000
    given = torch.zeros((m, k), device="cuda").to(E4M3)
    assert mk.quantize_fp8(torch.ones((m, k), dtype=BF16, device="cuda"), codes=given)[0] is given
