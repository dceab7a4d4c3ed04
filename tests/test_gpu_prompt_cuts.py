"""``paged_prompt_attention`` where the work of a sequence is shared by CTAs and joined, against its definition in 64 bits
element by element: with and without a list of tasks, and values whose sums over the parts pass fp32's largest."""
import math

import pytest
import torch

import prompt_util as P
import serving_util as U
from test_gpu_prompt_attention import _cache, _check, _run

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# few sequences find their tasks themselves; more than 32, or more than two items an SM (20 sequences of 16 kv heads), from a list
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("new,lengths,hq,hkv,d", [([4], [7000], 4, 2, 64), ([300, 40, 1, 0, 200], [1300, 3040, 6, 70, 200], 4, 2, 64),
                                                  ([4, 1, 200] + [0, 3] * 18 + [90], [7004, 2501, 3200] + [9, 3] * 18 + [5090], 4, 2, 64),
                                                  ([1, 0, 30] + [2] * 37, [6001, 4, 3030] + [150] * 37, 4, 2, 128),
                                                  ([5, 60] + [1] * 18, [5005, 3000] + [200] * 18, 16, 16, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2500, 4)])
def test_cut_sequences(new, lengths, hq, hkv, d, cache, window, sinks):
    _check(new, lengths, hq, hkv, d, 16, cache, window, sinks, seed=len(new))


@pytest.mark.parametrize("starts,lengths", [([0, 150, 300, 100, 80, 80], [5000, 3000, 900, 900, 900]), ([0, 150, 300, 500, 400, 380], [5000, 3000, 900, 900, 900]),
                                            ([0, 150, 300, 300, 300, 300], [5000, 3000, -1, 7000, 2 ** 31 - 1])])
@pytest.mark.parametrize("empty", [0, 40])
def test_cut_sequences_among_starts_that_decrease(starts, lengths, empty):
    kc, vc, table, _, _ = _cache([5000, 3000] + [1000] * 3 + [1] * empty, 2, 64, 16, BF16, 22)
    q = torch.randn((400, 4, 64), generator=torch.Generator().manual_seed(22)).to(BF16)
    st, ln = torch.tensor(starts + starts[-1:] * empty, dtype=torch.int32), torch.tensor(lengths + [1] * empty, dtype=torch.int32)
    out, lse, status = _run(q, kc, vc, table, st, ln)
    assert status == (-10 if min(starts[2:]) < 300 or max(starts) > 400 else 0)
    want, wl, err, el = P.prompt_attention(q[:300], kc, vc, table, torch.tensor([0, 150, 300]), ln[:2], 64 ** -0.5)
    # (rows below 100 are not those of a sequence whose starts decrease to them)
    U.assert_within(out[:300], want, U.half_step(BF16, want) + err, "out")
    U.assert_within(lse[:300], wl, el, "lse")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("among", [0, 40])
def test_parts_of_large_values(d, among):
    # one dominating weight of the same size in several parts, each times 2e38: the sum of two is past fp32's largest, the
    # result is not.  (Parts whose own sums are past it are worked on again by themselves.)
    n, big = 7000, float(torch.tensor(2e38).to(BF16))
    kc, vc, table, _, _ = _cache([n] + [1] * among, 2, d, 16, BF16, 3)
    kc = kc * 0.01
    at = torch.tensor([100, 1500, 2900, 4300, 5700, 6900])
    pages = table[0, at // 16].long()
    kc[pages, :, at % 16] = 40.0 / d ** 0.5
    vc[pages, :, at % 16] = torch.where(torch.arange(d) % 3 == 0, -big, big).to(BF16)
    q = torch.ones((4 + among, 4, d), dtype=BF16)
    st = torch.tensor([0, 4] + [4 + i for i in range(1, among + 1)], dtype=torch.int32)
    ln = torch.tensor([n] + [1] * among, dtype=torch.int32)
    out, lse, status = _run(q, kc, vc, table, st, ln)
    want, wl, err, el = P.prompt_attention(q[:4], kc, vc, table, st[:2], ln[:1], d ** -0.5)
    assert status == 0 and torch.isfinite(want).all()
    U.assert_within(out[:4], want, U.half_step(BF16, want) + err, "out")
    U.assert_within(lse[:4], wl, el, "lse")


@pytest.mark.parametrize("among", [0, 40])
@pytest.mark.parametrize("where", [100, 6900])
def test_an_infinity_whose_part_has_no_weight(among, where):
    # a visible infinity is the result however small its weight: as in a sequence that is not cut
    n, d = 7000, 64
    kc, vc, table, _, _ = _cache([n] + [1] * among, 2, d, 16, BF16, 4)
    kc = kc * 0.01
    for at, score in ((3500, 60.0), (where, -150.0)):
        kc[table[0, at // 16].long(), :, at % 16] = score / d ** 0.5
    first, last = where // 1024 * 1024, (where // 1024 + 1) * 1024
    for at in range(max(0, first - 1024), min(n, last + 1024)):  # (and of its neighbours: nothing in the part weighs anything)
        if at != 3500:
            kc[table[0, at // 16].long(), :, at % 16] = -150.0 / d ** 0.5
    vc[table[0, where // 16].long(), :, where % 16, 5] = math.inf
    vc[table[0, where // 16].long(), 1, where % 16, 7] = -math.inf
    q = torch.ones((4 + among, 4, d), dtype=BF16)
    st = torch.tensor([0, 4] + [4 + i for i in range(1, among + 1)], dtype=torch.int32)
    out, lse, status = _run(q, kc, vc, table, st, torch.tensor([n] + [1] * among, dtype=torch.int32))
    want, wl, err, el = P.prompt_attention(q[:4], kc, vc, table, st[:2], torch.tensor([n]), d ** -0.5)
    assert status == 0 and (want[:, :, 5] == math.inf).all() and (want[:, 2:, 7] == -math.inf).all()
    U.assert_within(out[:4], want, U.half_step(BF16, want) + err, "out")
    U.assert_within(lse[:4], wl, el, "lse")
