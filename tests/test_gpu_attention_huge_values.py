"""``paged_attention`` with finite keys and values up to bf16's largest: tokens
without weight, query elements of zero, and rows whose values are all of that
size (the weighted sum stays in range although the sum before its division by
the weights' would not)."""
import numpy as np
import pytest
import torch

import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32 = torch.bfloat16, torch.float32
LARGEST = torch.finfo(BF16).max


def _call(q, k, v, lengths, page=16, width=None):
    """One call over sequences of dense keys and values [row][kv head][token][d], checked against the definition."""
    n, hkv, _, d = k.shape
    table, total = U.pages(lengths, page, np.random.default_rng(0))
    kc, vc = (torch.full((total, hkv, page, d), float("nan"), dtype=BF16) for _ in range(2))
    for b, length in enumerate(lengths):
        for p in range(length):
            at = int(table[b, p // page]), slice(None), p % page
            kc[at], vc[at] = k[b, :, p], v[b, :, p]
    if width:
        table = torch.cat([table, torch.full((n, width), -1, dtype=torch.int32)], 1)
    lens = torch.tensor(lengths, dtype=torch.int32)
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = mk.paged_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), lse=lse)
    want, wlse, err, lerr = U.attention(q, kc, vc, table, lens, d ** -0.5)
    U.assert_within(out, want, U.half_step(q.dtype, want) + err, "out")
    U.assert_within(lse, wlse, lerr, "lse")


def _inputs(rows, tokens, x, seed, hq=4, hkv=2, d=128):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((rows, hq, d), generator=g).abs().add(0.5).to(x)
    k, v = (torch.randn((rows, hkv, tokens, d), generator=g).to(BF16) for _ in range(2))
    return q, k, v


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("huge", [1e33, 1e36, LARGEST, -LARGEST])
@pytest.mark.parametrize("lengths,width", [([40], None), ([40, 17], None), ([1500, 900], 300)])   # a cluster, whole rows, cut rows
def test_values_of_tokens_without_weight(x, huge, lengths, width):
    q, k, v = _inputs(len(lengths), max(lengths), x, 1)
    v.fill_(1.0)
    for p in (3, 12):
        k[:, :, p] = -40.0                                  # scores below -200: e to that is no fp32 number
        v[:, :, p] = huge
    _call(q, k, v, lengths, width=width)


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("huge", [1e36, LARGEST])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_against_query_elements_of_zero(x, huge, d):
    q, k, v = _inputs(2, 50, x, 2, d=d)
    q[:, :, 5], q[:, :, d - 1] = 0.0, -0.0
    k[:, :, :, 5], k[:, :, ::3, d - 1] = huge, -huge
    _call(q, k, v, [50, 33])


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("lengths,width", [([1], None), ([300], None), ([300, 77, 1], None), ([2500, 40, 1200], 300)])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (2, 2, 64), (16, 1, 128)])
def test_rows_of_the_largest_values(x, lengths, width, hq, hkv, d):
    q, k, v = _inputs(len(lengths), max(lengths), x, 3, hq, hkv, d)
    q, k = q * 0.1, k * 0.1                                 # every token has weight
    v.fill_(LARGEST)
    v[:, :, :, 1::2] = -LARGEST
    v[:, :, ::2, 3] *= -1.0                                 # and one element whose sum cancels
    _call(q.to(x), k, v, lengths, width=width)
