"""The README's examples of the serving operators, run as they stand."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

pytest.importorskip("persistent_transformer_megakernel_gb300")

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_a_step_takes_pages_that_no_sequence_has():
    with open(README) as f:
        blocks = [b for b in re.findall(r"```python\n(.*?)```", f.read(), flags=re.S) if "mk.paged_" in b]
    assert len(blocks) == 2
    names = {}
    exec(blocks[0], names)
    out = names["out"]
    assert out.shape == (4, 16, 128) and torch.isfinite(out[:3]).all()
    exec(blocks[1], names)
    page, table, lengths, totals, free, used = (names[n].cpu() if torch.is_tensor(names[n]) else names[n]
                                                for n in ("page", "table", "lengths", "totals", "free", "used"))
    assert totals.tolist() == [300, 901, 80, 0] and used.item() == 19 + 0 + 4
    held = [int(p) for i, n in enumerate(lengths.tolist()) for p in table[i, :-(-n // page)]]
    assert not set(held) & set(free.tolist())
    now = [int(p) for i, n in enumerate(totals.tolist()) for p in table[i, :-(-n // page)]]
    assert len(set(now)) == len(now) == 19 + 57 + 5
    assert torch.isfinite(names["out"][:365].float()).all() and torch.isfinite(names["logits"]).all()
