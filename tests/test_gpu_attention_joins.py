"""``paged_attention`` of rows that many CTAs share, so that their parts are joined
in more than one chunk of 32: a long row with a short one beside it on few kv
heads (a single row goes to clusters instead)."""
import numpy as np
import pytest
import torch

import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _cache(tokens, hkv, d, cache, page, seed):
    """Random pages for a sequence of ``tokens`` and a short one: keys, values, page table, scales."""
    g = torch.Generator().manual_seed(seed)
    table, total = U.pages([tokens, 100], page, np.random.default_rng(seed))
    unit = 40.0 if cache == E4M3 else 1.0
    kc, vc = ((torch.randn((total, hkv, page, d), generator=g) * unit).to(cache) for _ in range(2))
    scales = [torch.rand(hkv, generator=g) * 0.02 + 0.015 for _ in range(2)] if cache == E4M3 else [None, None]
    return kc, vc, table, scales


def _check(q, kc, vc, table, scales, lengths, window=0):
    lens = torch.tensor(lengths, dtype=torch.int32)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = mk.paged_attention(dev(q), dev(kc), dev(vc), dev(table), dev(lens), window=window, k_scale=dev(scales[0]), v_scale=dev(scales[1]), lse=lse)
    want, wlse, err, lerr = U.attention(q, kc, vc, table, lens, q.shape[2] ** -0.5, window, *scales)
    U.assert_within(out, want, U.half_step(q.dtype, want) + err, "%s out" % lengths)
    U.assert_within(lse, wlse, lerr, "%s lse" % lengths)


# tiles are 16 slots, 32 over an e4m3 cache or for heads of 64; a CTA has 16 of them or more
@pytest.mark.parametrize("x,cache,hq,hkv,d,lengths", [
    (BF16, BF16, 2, 1, 128, [20011, 5]),                    # 79 CTAs
    (F32, BF16, 4, 1, 128, [20011, 0]),
    (BF16, BF16, 16, 1, 128, [20011, 100]),                 # 16 query heads: two blocks of columns, two CTAs a join
    (F32, E4M3, 2, 1, 128, [40022, 5]),
    (BF16, E4M3, 16, 1, 64, [40022, 5]),
    (BF16, BF16, 2, 2, 64, [40022, 64]),                    # all CTAs, two kv heads
    (BF16, BF16, 40, 1, 128, [30000, 1]),                   # three blocks of query heads
])
def test_rows_of_many_parts(x, cache, hq, hkv, d, lengths):
    kc, vc, table, scales = _cache(lengths[0], hkv, d, cache, 16, 1)
    q = (torch.randn((2, hq, d), generator=torch.Generator().manual_seed(2)) * 1.5).to(x)
    _check(q, kc, vc, table, scales, lengths)
    _check(q.flip(0), kc, vc, table.flip(0), scales, lengths[::-1])
    _check(q, kc, vc, table, scales, lengths, window=lengths[0] - 7)


@pytest.mark.parametrize("around", [32, 64, 96])
def test_rows_about_a_whole_number_of_chunks(around):
    # a CTA takes 16 units of work: rows of one tile less to some more than `around` CTAs' share
    tokens = (around + 2) * 16 * 16
    kc, vc, table, scales = _cache(tokens, 1, 128, BF16, 16, 3)
    q = torch.randn((2, 1, 128), generator=torch.Generator().manual_seed(4))
    for tiles in range((around - 1) * 16 - 4, (around + 1) * 16 + 4, 3):
        _check(q, kc, vc, table, scales, [tiles * 16 - 5, 33])
