"""Sizes near 2^31 that the C entry points of a step's operators refuse before any CUDA call: loops over them would pass
32 bits (no GPU; the pointers are never followed)."""
import ctypes as C
import os

import pytest

import persistent_transformer_megakernel_gb300 as mk
from persistent_transformer_megakernel_gb300 import _binding as B

if not os.path.exists(mk.lib_path()):
    from persistent_transformer_megakernel_gb300 import build
    build.build()

MOST = 2 ** 31 - 1
UNSUPPORTED = -2


@pytest.mark.parametrize("far", [MOST, MOST - 1000, MOST - 5000])
def test_histories_and_biases(far):
    lib = mk.load_library()

    def logits(**f):
        a = dict(n=1, vocab=8, dtype=0, x=16, out=16, x_row=8, out_row=8, tokens=16, bias_ids=16, bias=16)
        return lib.mk_adjust_logits(C.byref(B.mk_logits_args(**{**a, **f})), None)
    assert logits(vocab=far) == UNSUPPORTED
    assert logits(columns=far) == UNSUPPORTED
    assert logits(biases=far) == UNSUPPORTED
    assert logits(n=0, columns=far) == 0


@pytest.mark.parametrize("rows", [MOST, MOST - 65536, MOST - 131072])
def test_rows_of_a_plan(rows):
    # as many pages as rows are taken where a page has one token, in steps of all threads of the device
    a = B.mk_plan_args(n=2, rows=rows, page_size=1, lengths=16, counts=16, table=16, table_cols=MOST, table_stride=MOST, free=16, free_count=MOST, used=16,
                       seqs=16, slots=16, starts=16, totals=16, used_out=16)
    assert mk.load_library().mk_paged_plan(C.byref(a), None) == UNSUPPORTED
