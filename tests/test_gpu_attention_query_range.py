"""``paged_attention`` over an 8-bit cache with queries of elements of very
different size: an element is rounded to 2^-38 of its head's largest, no more is
lost, whatever the keys beside the largest hold."""
import numpy as np
import pytest
import torch

import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 20, 2.0 ** 28, 2.0 ** 34])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (16, 1, 64)])
def test_an_outlier_against_keys_of_zero(x, ratio, hq, hkv, d):
    g = torch.Generator().manual_seed(0)
    lengths = [70, 5, 300]
    table, total = U.pages(lengths, 16, np.random.default_rng(0))
    kc, vc = ((torch.randn((total, hkv, 16, d), generator=g) * 40).to(E4M3) for _ in range(2))
    kc[..., 11] = 0.0
    ks, vs = (torch.rand(hkv, generator=g) * 0.02 + 0.015 for _ in range(2))
    q = torch.randn((3, hq, d), generator=g).to(x)
    q[:, :, 11] = ratio
    lens = torch.tensor(lengths, dtype=torch.int32)
    lse = torch.zeros((3, hq), device="cuda")
    out = mk.paged_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), k_scale=ks.cuda(), v_scale=vs.cuda(), lse=lse)
    want, wlse, err, lerr = U.attention(q, kc, vc, table, lens, d ** -0.5, 0, ks, vs)
    # what the queries' rounding adds to a score: 2^-38 of the largest element times a key's sum of absolute values; twice
    # that on a weight (its own score's and the sum's), times the weighted sum of absolute values, which is at most the largest
    for b, n in enumerate(lengths):
        k = U.gather(kc, table[b], n) * ks.to(U.F64)[:, None, None]
        v = U.gather(vc, table[b], n) * vs.to(U.F64)[:, None, None]
        s = (k.abs().sum(-1).amax(-1) * ratio * 2.0 ** -38 * d ** -0.5).repeat_interleave(hq // hkv)
        err[b] += (torch.expm1(2 * s) * v.abs().amax((1, 2)).repeat_interleave(hq // hkv))[:, None]
        lerr[b] += s
    U.assert_within(out, want, U.half_step(x, want) + err, "out")
    U.assert_within(lse, wlse, lerr, "lse")
