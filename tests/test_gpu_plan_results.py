"""The results that ``paged_plan`` makes beside those that it is given."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")


def z(*s):
    return torch.zeros(s, dtype=torch.int32, device="cuda")


# every choice of results that are given, for steps without sequences, without rows and with both
@pytest.mark.parametrize("n,rows", [(0, 0), (0, 3), (2, 0), (2, 5)])
def test_some_are_given(n, rows):
    names, sizes = ("seqs", "slots", "starts", "totals", "used_out"), (rows, rows, n + 1, n, 1)
    counts = torch.tensor([0, rows][:n], dtype=torch.int32, device="cuda")
    want = [t.tolist() for t in mk.paged_plan(z(n), z(n, 2), torch.tensor([4, 5, 6], dtype=torch.int32, device="cuda"), z(1), 16, counts=counts, rows=rows)]
    for k in range(6):
        for some in itertools.combinations(range(5), k):
            given = {names[i]: z(sizes[i]) for i in some}
            got = mk.paged_plan(z(n), z(n, 2), torch.tensor([4, 5, 6], dtype=torch.int32, device="cuda"), z(1), 16, counts=counts, rows=rows, **given)
            assert [t.tolist() for t in got] == want
            assert all(got[i] is given[names[i]] for i in some)
