"""Prompts among whose first tokens are values or keys that are no numbers: every row behind them is worked on again."""
import math

import pytest
import torch

import prompt_util as P
import serving_util as U
from test_gpu_prompt_attention import _cache, _run

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,count,page,window,sinks", [(1500, 1500, 16, 0, 0), (1500, 1500, 16, 700, 40), (3000, 37, 7, 0, 0), (2600, 300, 24, 1111, 9)])
def test_a_value_among_the_first_tokens(n, count, page, window, sinks, d, cache):
    kc, vc, table, ks, vs = _cache([n], 2, d, page, cache, 8)
    raw = vc.view(torch.uint8) if cache == E4M3 else vc
    raw[table[0, 3 // page], 1, 3 % page, 5] = 0x7F if cache == E4M3 else math.nan
    if cache == BF16:
        vc[table[0, 3 // page], 0, 3 % page, 9] = -math.inf
    q = torch.randn((count, 4, d), generator=torch.Generator().manual_seed(3)).to(BF16)
    starts, ln = torch.tensor([0, count], dtype=torch.int32), torch.tensor([n], dtype=torch.int32)
    out, lse, status = _run(q, kc, vc, table, starts, ln, window, sinks, ks, vs)
    want, wl, err, el = P.prompt_attention(q, kc, vc, table, starts, ln, d ** -0.5, window, sinks, ks, vs)
    hit = P.seen(n, n - count, n, window, sinks)[:, 3]
    assert status == 0 and hit.any() and torch.isnan(want[hit][:, 2:, 5]).all() and int((~torch.isfinite(want)).sum()) == int(hit.sum()) * (4 if cache == BF16 else 2)
    U.assert_within(out, want, U.half_step(BF16, want) + err, "out")
    U.assert_within(lse, wl, el, "lse")


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("n,count,window", [(1500, 1500, 0), (3000, 37, 0), (2600, 300, 1111)])
def test_a_key_among_the_first_tokens(n, count, window, cache):
    kc, vc, table, ks, vs = _cache([n], 2, 64, 16, cache, 9)
    good = _run(torch.ones((count, 4, 64), dtype=BF16), kc, vc, table, torch.tensor([0, count], dtype=torch.int32), torch.tensor([n], dtype=torch.int32), window, 4, ks, vs)
    at = n - count + 20 if window == 0 else 2
    raw = kc.view(torch.uint8) if cache == E4M3 else kc
    raw[table[0, at // 16], 1, at % 16, 0] = 0x7F if cache == E4M3 else math.nan
    out, lse, status = _run(torch.ones((count, 4, 64), dtype=BF16), kc, vc, table, torch.tensor([0, count], dtype=torch.int32), torch.tensor([n], dtype=torch.int32), window, 4, ks, vs)
    first = max(0, at - (n - count))
    assert status == 0 and torch.isnan(out[first:, 2:]).all() and torch.isnan(lse[first:, 2:]).all()
    assert torch.equal(out[:first], good[0][:first]) and torch.equal(out[:, :2], good[0][:, :2]) and torch.equal(lse[:, :2], good[1][:, :2])
