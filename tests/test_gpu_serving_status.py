"""``check_status`` waits for the operator whose error it reports, on whichever stream that ran."""
import pytest
import torch

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16 = torch.bfloat16


def _busy(a):
    for _ in range(40):                                     # some tens of milliseconds
        a = a @ a * 1e-3
    return a


@pytest.mark.parametrize("op", ["append", "attention"])
def test_an_error_on_a_side_stream(op):
    kc, vc = (torch.zeros((2, 1, 4, 64), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.full((1, 2), 99, dtype=torch.int32, device="cuda")                # a page that is none
    x = torch.ones((1, 1, 64), dtype=BF16, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    a = torch.randn((6144, 6144), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _busy(a)                                            # (the libraries' first calls are slow)
    for _ in range(2):
        status.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            _busy(a)
        if op == "append":
            mk.paged_append(x, x, kc, vc, table, one, status=status, stream=side)
        else:
            mk.paged_attention(x, kc, vc, table, one, status=status, stream=side)
        with pytest.raises(mk.MKError) as e:
            mk.check_status(status, stream=side)
        assert e.value.code == -10
    status.zero_()
    torch.cuda.synchronize()
    table.zero_()
    mk.paged_append(x, x, kc, vc, table, one, status=status, stream=torch.cuda.current_stream())
    mk.check_status(status, stream=torch.cuda.current_stream())
    mk.check_status(status)


def test_out_of_memory_is_torchs_own_error():
    # the result of this call is 34 GB, which the process is not allowed; nothing of that size exists
    n = 1 << 20
    kc = torch.zeros((1, 64, 4, 128), dtype=BF16, device="cuda")
    q = torch.zeros((1, 64, 128), device="cuda").expand(n, -1, -1)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda").expand(n, -1)
    lengths = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.set_per_process_memory_fraction(0.02)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            mk.paged_attention(q, kc, kc, table, lengths)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    out = mk.paged_attention(q[:2], kc, kc, table[:2], lengths[:2] + 2)
    assert (out == 0).all()
