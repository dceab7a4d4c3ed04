"""Starts that decrease again and again, so that their sequences promise more tasks than 2^31: refused as bad."""
import pytest
import torch

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16 = torch.bfloat16


def test_more_tasks_than_32_bits_hold():
    # 8192 sequences of the same 1310720 rows, each 5120 items of 64 heads: 2.7e9
    n, rows, heads, d = 16384, (1 << 20) + (1 << 18), 64, 64
    kc, vc = (torch.zeros((1, heads, 16, d), dtype=BF16, device="cuda") for _ in range(2))
    starts = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    starts[1::2] = rows
    q = torch.zeros((1, heads, d), dtype=BF16, device="cuda").expand(rows, -1, -1)
    out = torch.full((rows, heads, d), 7.0, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table, lengths = torch.zeros((n, 20), dtype=torch.int32, device="cuda"), torch.full((n,), 5, dtype=torch.int32, device="cuda")
    mk.paged_prompt_attention(q, kc, vc, table, starts, lengths, out=out, status=status)
    with pytest.raises(mk.MKError) as e:
        mk.check_status(status)
    assert e.value.code == -10 and (out == 7).all()
