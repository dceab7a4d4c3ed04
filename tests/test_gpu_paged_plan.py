"""``paged_plan`` against the plan made token by token."""
import random

import pytest
import torch

import prompt_util as P

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(rng, n, page, hi, hi_new, step):
    lengths = [rng.choice([-1, -7, 0, page, rng.randint(0, hi), rng.randint(0, hi)]) for _ in range(n)]
    counts = None if step else [rng.choice([0, 1, -3, page, rng.randint(0, hi_new)]) for _ in range(n)]
    cols = -(-(hi + page + (1 if step else hi_new)) // page) + 1
    table = [[rng.randint(-1, 99) for _ in range(cols)] for _ in range(n)]
    take = sum((1 if step else max(0, counts[i])) if lengths[i] >= 0 else 0 for i in range(n))
    free = random.Random(1).sample(range(1000, 1000 + take + 2 * n + 20), take + 2 * n + 10)
    return lengths, counts, table, free, take


def _check(got, table, want, status):
    seqs, slots, starts, totals, used, grid, fits = want
    for g, w in zip(got, (seqs, slots, starts, totals, [used])):
        assert g.tolist() == w
    assert table.tolist() == grid
    assert int(status) == (0 if fits else -3)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("n,page,hi,hi_new", [(1, 16, 40, 70), (2, 1, 5, 9), (7, 24, 300, 100), (33, 100, 9, 3), (600, 16, 900, 60),
                                              (5, 16, 100, 40000)])
def test_plans(n, page, hi, hi_new, step):
    rng = random.Random(n * 31 + page)
    lengths, counts, table, free, take = _case(rng, n, page, hi, hi_new, step)
    for rows in ((n,) if step else (take, take + 13)):
        t, s = i32(table), torch.zeros(1, dtype=torch.int32, device="cuda")
        got = mk.paged_plan(i32(lengths), t, i32(free), i32([3]), page, counts=None if step else i32(counts), rows=rows, status=s)
        _check(got, t, P.plan(lengths, counts, table, free, 3, page, rows), s)


def test_no_sequences():
    t, s = torch.zeros((0, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = mk.paged_plan(none, t, none, i32([5]), 16, counts=none, rows=6, status=s)
    assert [g.tolist() for g in got] == [[-1] * 6, [-1] * 6, [0], [], [5]] and int(s) == 0
    assert [g.tolist() for g in mk.paged_plan(none, t, none, i32([5]), 16)] == [[], [], [0], [], [5]]


@pytest.mark.parametrize("short", ["rows", "pages", "columns", "length", "used"])
def test_a_step_that_does_not_fit_is_not_made(short):
    lengths, counts, page = [30, -1, 16, 5], [10, 4, 1, 0], 16        # three pages: 10 tokens end in a third, the 17th opens one
    cols, free, rows, used = 3, [7, 8, 9, 10], 12, 2
    if short == "rows":
        rows = 10
    elif short == "pages":
        used = 3
    elif short == "columns":
        cols = 2
    elif short == "used":
        used = -1
    else:
        lengths = [30, -1, 2 ** 31 - 1, 5]
    table = [[1] * cols for _ in lengths]
    t, s = i32(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mk.paged_plan(i32(lengths), t, i32(free), i32([used]), page, counts=i32(counts), rows=rows, status=s)
    assert [g.tolist() for g in got] == [[-1] * rows, [-1] * rows, [0] * 5, lengths, [used]]
    assert t.tolist() == table
    with pytest.raises(mk.MKError):
        mk.check_status(s)


def test_in_place_strided_and_captured():
    # a decode loop of captured steps: totals are lengths, used_out is used, the table is part of a wider one
    n, page, steps = 70, 8, 20
    rng = random.Random(5)
    lengths = [rng.choice([-1, 0, 7, 8, rng.randint(0, 60)]) for _ in range(n)]
    free = list(range(500, 500 + 4 * n))
    wide = torch.full((n + 2, 40), -5, dtype=torch.int32, device="cuda")
    table = wide[:n, 3:20]
    ln, used, s = i32(lengths), i32([1]), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = dict(seqs=i32([0] * n), slots=i32([0] * (n + 1))[1:], starts=i32([0] * (n + 1)))
    f = i32(free)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mk.paged_plan(ln, table, f, used, page, totals=ln, used_out=used, status=s, **out)
    ln.copy_(i32(lengths)), used.fill_(1), table.fill_(-5)
    grid, at = [[-5] * 17 for _ in range(n)], 1
    for _ in range(steps):
        g.replay()
        seqs, slots, starts, lengths, at, grid, fits = P.plan(lengths, None, grid, free, at, page, n)
        assert fits and ln.tolist() == lengths and int(used) == at and out["slots"].tolist() == slots and out["seqs"].tolist() == seqs
        assert table.tolist() == grid
    assert (wide[:, :3] == -5).all() and (wide[:, 20:] == -5).all() and (wide[n:] == -5).all() and int(s) == 0


def test_many_sequences():
    n = 16384
    lengths, counts = torch.arange(n) % 50, (torch.arange(n) * 7) % 5
    t, s = torch.full((n, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = int(counts.sum())
    seqs, slots, starts, totals, used = mk.paged_plan(lengths.int().cuda(), t, torch.arange(2 * n, dtype=torch.int32, device="cuda"), i32([0]), 16,
                                                      counts=counts.int().cuda(), rows=rows, status=s)
    assert int(s) == 0
    assert torch.equal(seqs.cpu().long(), torch.repeat_interleave(torch.arange(n), counts))
    assert torch.equal(starts.cpu()[1:].long(), counts.cumsum(0)) and torch.equal(totals.cpu().long(), lengths + counts)
    assert torch.equal(slots.cpu().long(), torch.arange(rows) - (counts.cumsum(0) - counts)[seqs.cpu().long()] + lengths[seqs.cpu().long()])
    new = (lengths + counts + 15) // 16 - (lengths + 15) // 16
    assert int(used) == int(new.sum()) and sorted(t.cpu()[t.cpu() >= 0].tolist()) == list(range(int(used)))
    with pytest.raises(mk.MKError):
        mk.paged_plan(torch.zeros(n + 1, dtype=torch.int32, device="cuda"), torch.zeros((n + 1, 1), dtype=torch.int32, device="cuda"), i32([0]), i32([0]), 16)
