"""What the serving operators write counts as changed: an autograd graph that has
saved it does not use it unnoticed."""
import pytest
import torch

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16 = torch.bfloat16


def _tensors():
    kc, vc = (torch.zeros((2, 1, 4, 64), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    x = torch.ones((1, 1, 64), dtype=BF16, device="cuda")
    return kc, vc, table, x, torch.ones(1, dtype=torch.int32, device="cuda")


def test_versions_grow():
    kc, vc, table, x, one = _tensors()
    q_out, out, lse, status = torch.zeros_like(x), torch.zeros_like(x), torch.zeros((1, 1), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    written = (kc, vc, q_out, status)
    before = [t._version for t in written + (x, table, one)]
    mk.paged_append(x, x, kc, vc, table, one, q=x, q_out=q_out, status=status)
    assert [t._version for t in written] == [v + 1 for v in before[:4]]
    before2 = [t._version for t in (out, lse, status, kc, vc)]
    mk.paged_attention(q_out, kc, vc, table, one, out=out, lse=lse, status=status)
    assert [t._version for t in (out, lse, status)] == [v + 1 for v in before2[:3]]
    y = torch.zeros((1, 8), device="cuda")
    codes, scales = torch.zeros((8, 32), dtype=torch.uint8, device="cuda"), torch.ones((8, 1), dtype=BF16, device="cuda")
    v = y._version
    mk.matvec_q4(torch.ones((1, 64), device="cuda"), codes, scales, out=y)
    assert y._version == v + 1
    assert [t._version for t in (kc, vc)] == before2[3:] and [t._version for t in (x, table, one)] == before[4:]


def test_a_saved_output_that_is_overwritten():
    kc, vc, table, x, one = _tensors()
    out = torch.zeros_like(x)
    a = torch.ones_like(x, requires_grad=True)
    loss = (a * out).sum()                                  # saves out
    mk.paged_attention(x, kc, vc, table, one, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    view = kc[0]
    loss = (a * view[:, :1]).sum()
    mk.paged_append(x, x, kc, vc, table, one)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors():
    with torch.inference_mode():
        kc, vc, table, x, one = _tensors()
        q = mk.paged_append(x, x, kc, vc, table, one, q=x)
        out = torch.empty_like(x)
        mk.paged_attention(q, kc, vc, table, one, out=out)
    mk.paged_attention(q, kc, vc, table, one, out=out)
    mk.paged_append(x, x, kc, vc, table, one, q=x, q_out=q)
    torch.cuda.synchronize()
    assert torch.equal(q, x) and torch.isfinite(out).all()
