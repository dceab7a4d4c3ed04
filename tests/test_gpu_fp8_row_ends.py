"""``matmul_fp8`` into rows that end anywhere in a larger buffer: what is behind them stays."""
import pytest
import torch

import prompt_util as P
import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("residual", [None, "apart", "in place"])
@pytest.mark.parametrize("m,k", [(1, 32), (1, 2048), (3, 48), (40, 1024), (200, 272)])
@pytest.mark.parametrize("n", [1, 2, 5, 46, 58, 61, 64, 126, 129, 1001, 2322])
def test_rows_on_16_bytes(n, m, k, residual, dtype):
    g = torch.Generator().manual_seed(n * m)
    x, w = torch.randn((m, k), generator=g).to(BF16).cuda(), torch.randn((n, k), generator=g).cuda()
    c, s = mk.quantize_fp8(x)
    cw, sw = mk.quantize_fp8_weight(w)
    unit = 128 // torch.finfo(dtype).bits
    wide = -(-n // unit) * unit + unit
    room = torch.full((m + 2, wide), 7.0, dtype=dtype, device="cuda")
    out, r = room[1:m + 1, :n], torch.randn((m, wide), generator=g).to(dtype).cuda()[:, :n]
    if residual == "in place":
        out.copy_(r)
    mk.matmul_fp8(c, s, cw, sw, out=out, residual=None if residual is None else out if residual == "in place" else r)
    want, err = P.product(c.cpu(), s.cpu(), cw.cpu(), sw.cpu())
    if residual:
        want, err = want + r.cpu().double(), err + (want.abs() + r.cpu().double().abs()) * 2.0 ** -24
    U.assert_within(out, want, U.half_step(dtype, want) + err, "y")
    assert (room[0] == 7).all() and (room[-1] == 7).all() and (room[:, n:] == 7).all()
