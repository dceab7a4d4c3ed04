"""Serving operators have no forward-mode derivative: a tensor with a tangent is refused (no GPU)."""
import os

import pytest
import torch
import torch.autograd.forward_ad as fwd

import persistent_transformer_megakernel_gb300 as mk
from persistent_transformer_megakernel_gb300 import serving as S

BF16 = torch.bfloat16

if not os.path.exists(mk.lib_path()) or not os.path.exists(os.path.join(os.path.dirname(mk.lib_path()), "_mktorch.so")):
    from persistent_transformer_megakernel_gb300 import build
    build.build()


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def calls():
    m = S.native()
    kc, vc, table = torch.zeros((6, 2, 16, 64), dtype=BF16), torch.zeros((6, 2, 16, 64), dtype=BF16), i32(3, 4)
    w, ws = mk.quantize_fp8_weight(torch.zeros((8, 128)))
    x = torch.zeros((3, 4, 64), dtype=BF16)
    return [(x, lambda t: m.check_prompt(t, kc, vc, table, i32(4), i32(3))),
            (x, lambda t: m.check_attention(t, kc, vc, table, i32(3))),
            (kc, lambda t: m.check_attention(x, t, vc, table, i32(3))),
            (x[:, :2], lambda t: m.check_append(t, x[:, :2], kc, vc, table, i32(3))),
            (torch.ones((1, 64)), lambda t: m.check_matvec(t, torch.zeros((8, 32), dtype=torch.uint8), torch.ones((8, 1), dtype=BF16))),
            (torch.zeros((3, 128), dtype=BF16), lambda t: m.check_quantize(t)),
            (torch.zeros((3, 1)), lambda t: m.check_matmul(torch.zeros((3, 128)).to(w.dtype), t, w, ws)),
            (torch.zeros((3, 100)), lambda t: m.check_logits(t)),
            (torch.zeros((3, 2)), lambda t: m.check_logits(torch.zeros((3, 100)), bias_ids=i32(3, 2), bias=t))]


def test_tangents_are_refused():
    for plain, f in calls():
        f(plain)
        with fwd.dual_level():
            dual = fwd.make_dual(plain, torch.ones_like(plain))
            with pytest.raises(ValueError, match="tangent"):
                f(dual)
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):    # (which leaves forward mode on)
                f(dual)
            f(fwd.unpack_dual(dual).primal)
            f(plain)
        with torch.inference_mode():
            f(plain)
