"""Dispatch modes and the profiler see the results that serving operators make."""
import pytest
import torch
from torch.profiler import ProfilerActivity, profile
from torch.utils._python_dispatch import TorchDispatchMode

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16 = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls():
    g = torch.Generator().manual_seed(0)
    kc, vc = (torch.randn((4, 1, 16, 64), generator=g).to(BF16).cuda() for _ in range(2))
    q, table = torch.randn((5, 2, 64), generator=g).to(BF16).cuda(), torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    x = torch.randn((5, 256), generator=g).to(BF16).cuda()
    w = torch.randn((64, 256), generator=g).cuda()
    q4, w8, c = mk.quantize_q4(w), mk.quantize_fp8_weight(w), mk.quantize_fp8(x)
    starts, five, one, free, none = i32([0, 5]), i32([20]), i32([1]), i32([0, 1, 2]), i32([0])
    return [lambda: [mk.paged_append(q[:1, :1], q[:1, 1:], kc.clone(), vc.clone(), table, one, q=q[:1])],
            lambda: [mk.paged_attention(q[:1], kc, vc, table, five)], lambda: [mk.paged_prompt_attention(q, kc, vc, table, starts, five)],
            lambda: [mk.matvec_q4(x, *q4)], lambda: list(mk.quantize_fp8(x)), lambda: [mk.matmul_fp8(*c, *w8)],
            lambda: list(mk.paged_plan(one, table.clone(), free, none, 16)), lambda: [mk.adjust_logits(x, mask=torch.full((5, 8), -1, dtype=torch.int32, device="cuda"))]]


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in str(func):
            self.made.append(out.numel() * out.element_size())
        return out


def same(a, b):
    return all(x.dtype == y.dtype and torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x, y.view(torch.uint8) if y.element_size() == 1 else y)
               for x, y in zip(a, b))


def test_dispatch_modes():
    for i, f in enumerate(calls()):
        want = [t.clone() for t in f()]
        with Seen() as seen:
            got = f()
        assert same(got, want)
        assert sum(seen.made) >= sum(t.numel() * t.element_size() for t in got), (i, seen.made)


def test_the_profiler():
    for i, f in enumerate(calls()):
        want = [t.clone() for t in f()]
        with profile(activities=[ProfilerActivity.CPU]) as p:
            got = f()
        assert same(got, want)
        assert any(e.name.startswith("aten::empty") for e in p.events()), i


class Elsewhere(TorchDispatchMode):
    """New tensors on another device, or without memory."""

    def __init__(self, device):
        super().__init__()
        self.device = device

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        kwargs = dict(kwargs or {})
        if "empty" in str(func):
            kwargs["device"] = self.device
        return func(*args, **kwargs)


@pytest.mark.parametrize("device", ["meta", "cpu"])
def test_results_that_a_mode_puts_elsewhere(device):
    # (one call of each operator: the inputs are made before the mode)
    g = torch.Generator().manual_seed(0)
    kc, vc = (torch.randn((4, 1, 16, 64), generator=g).to(BF16).cuda() for _ in range(2))
    q, table = torch.randn((5, 2, 64), generator=g).to(BF16).cuda(), torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    x, mask = torch.randn((5, 256), generator=g).to(BF16).cuda(), torch.full((5, 8), -1, dtype=torch.int32, device="cuda")
    w = torch.randn((64, 256), generator=g).cuda()
    q4, w8, c = mk.quantize_q4(w), mk.quantize_fp8_weight(w), mk.quantize_fp8(x)
    starts, five, one, free, none = i32([0, 5]), i32([20]), i32([1]), i32([0, 1, 2]), i32([0])
    for f in (lambda: mk.paged_append(q[:1, :1], q[:1, 1:], kc, vc, table, one, q=q[:1]), lambda: mk.paged_attention(q[:1], kc, vc, table, five),
              lambda: mk.paged_prompt_attention(q, kc, vc, table, starts, five), lambda: mk.matvec_q4(x, *q4), lambda: mk.quantize_fp8(x),
              lambda: mk.matmul_fp8(*c, *w8), lambda: mk.paged_plan(one, table, free, none, 16), lambda: mk.adjust_logits(x, mask=mask)):
        with Elsewhere(device), pytest.raises(ValueError, match="without memory"):
            f()
