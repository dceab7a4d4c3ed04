"""Calls of the batched serving operators that are refused because their results
would not be what the call says (no GPU: the checks alone)."""
import os

import pytest
import torch

import persistent_transformer_megakernel_gb300 as mk
from persistent_transformer_megakernel_gb300 import _binding as B
from persistent_transformer_megakernel_gb300 import serving as S

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

if not os.path.exists(mk.lib_path()) or not os.path.exists(os.path.join(os.path.dirname(mk.lib_path()), "_mktorch.so")):
    from persistent_transformer_megakernel_gb300 import build
    build.build()


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _cache(**kw):
    return dict(dict(k_cache=torch.zeros((6, 2, 16, 64), dtype=BF16), v_cache=torch.zeros((6, 2, 16, 64), dtype=BF16), table=_i32(3, 4)), **kw)


def _append(**kw):
    a = dict(_cache(), k=torch.zeros((3, 2, 64)), v=torch.zeros((3, 2, 64)), slots=_i32(3), q=torch.zeros((3, 4, 64)))
    a.update(kw)
    return B.mk_append_args.from_buffer_copy(S.native().check_append(**a))


def _attention(**kw):
    a = dict(_cache(), q=torch.zeros((3, 4, 64)), lengths=_i32(3))
    a.update(kw)
    return B.mk_attention_args.from_buffer_copy(S.native().check_attention(**a))


def _matvec(**kw):
    a = dict(x=torch.zeros((3, 128)), codes=torch.zeros((10, 64), dtype=torch.uint8), scales=torch.zeros((10, 2), dtype=BF16))
    a.update(kw)
    return B.mk_matvec_q4_args.from_buffer_copy(S.native().check_matvec(**a))


def test_a_rotary_table_without_rows():
    assert _append(rope=torch.zeros((1, 32, 2))).rope
    for kw in (dict(), dict(positions=_i32(3)), dict(positions=_i32(3, 3), mrope_sections=(12, 10, 10))):
        with pytest.raises(ValueError, match="rope"):
            _append(rope=torch.zeros((0, 32, 2)), **kw)
