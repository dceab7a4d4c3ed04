"""Scales of an 8-bit cache that are no numbers, zero or negative, for prompts as for single tokens."""
import math

import pytest
import torch

import prompt_util as P
import serving_util as U
from test_gpu_prompt_attention import _cache, _run

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("n", [40, 3000])
def test_a_scale_of_one_head(n):
    count = 40
    kc, vc, table, ks, vs = _cache([n], 4, 64, 16, E4M3, 12)
    q = torch.randn((count, 8, 64), generator=torch.Generator().manual_seed(1)).to(BF16)
    starts, ln = torch.tensor([0, count], dtype=torch.int32), torch.tensor([n], dtype=torch.int32)
    good = _run(q, kc, vc, table, starts, ln, ks=ks, vs=vs)
    for which in (0, 1):
        bad = [ks.clone(), vs.clone()]
        bad[which][1] = math.nan
        out, lse, status = _run(q, kc, vc, table, starts, ln, ks=bad[0], vs=bad[1])
        assert status == 0 and torch.isnan(out[:, 2:4]).all()
        assert torch.equal(out[:, :2], good[0][:, :2]) and torch.equal(out[:, 4:], good[0][:, 4:])
        assert torch.equal(lse[:, :2], good[1][:, :2]) and torch.equal(lse[:, 4:], good[1][:, 4:])
        if which == 0:
            assert torch.isnan(lse[:, 2:4]).all()
        else:                                                # (worked out again, as the result is no number)
            _, wl, _, el = P.prompt_attention(q, kc, vc, table, starts, ln, 64 ** -0.5, 0, 0, ks, vs)
            U.assert_within(lse[:, 2:4], wl[:, 2:4], el[:, 2:4], "lse")
        one = mk.paged_attention(q[-1:].cuda(), kc.cuda(), vc.cuda(), table.cuda(), ln.cuda(), k_scale=bad[0].cuda(), v_scale=bad[1].cuda())
        assert torch.equal(torch.isnan(one[0]).cpu(), torch.isnan(out[-1]).cpu())
    # a negative scale turns the scores around, zero makes them alike
    ks[0], ks[3], vs[2] = -ks[0], 0.0, -vs[2]
    out, lse, status = _run(q, kc, vc, table, starts, ln, ks=ks, vs=vs)
    want, wl, err, el = P.prompt_attention(q, kc, vc, table, starts, ln, 64 ** -0.5, 0, 0, ks, vs)
    U.assert_within(out, want, U.half_step(BF16, want) + err, "out")
    U.assert_within(lse, wl, el, "lse")


def test_rows_that_see_nothing():
    kc, vc, table, ks, vs = _cache([3], 2, 64, 16, E4M3, 13)
    ks[:] = math.nan
    out, lse, status = _run(torch.ones((5, 4, 64), dtype=BF16), kc, vc, table, torch.tensor([0, 5], dtype=torch.int32), torch.tensor([3], dtype=torch.int32), ks=ks, vs=vs)
    assert status == 0 and (out[:2] == 0).all() and (lse[:2] == -math.inf).all() and torch.isnan(out[2:]).all()
