"""``matvec_q4`` where its launch is an unusual one: rows of which not one fits in
a CTA, many weights' rows beside them, many x rows, and x rows that fill each
number of column tiles."""
import pytest
import torch

import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32 = torch.bfloat16, torch.float32


def _run(m, n, k, group, x, zeros, only=None, seed=0):
    """One call; the outputs of the weights' rows ``only`` (all by default) are checked."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand((n, k // group), generator=g, device="cuda") + 0.2) * 0.01).to(BF16)
    z = torch.randint(0, 16, (n, k // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    xs = torch.randn((m, k), generator=g, device="cuda").to(x)
    res = torch.randn((m, n), generator=g, device="cuda").to(x)
    y = mk.matvec_q4(xs, codes, scales, zeros=z, residual=res)
    at = torch.arange(n) if only is None else torch.tensor(only)
    pick = lambda t: t[at.cuda()].cpu()  # noqa: E731
    w = U.dequantize(pick(codes), pick(scales), None if z is None else pick(z))
    xd, r = xs.cpu().to(U.F64), res.cpu().to(U.F64)[:, at]
    want = xd @ w.t()
    # a block's products: 16 chained sums at most; a multiply-add a block of 32 codes; the warps' and terms' sums
    err = (xd.abs() @ w.abs().t()) * ((16 + k / 32 + 32) * 2.0 ** -23)
    want = want + r
    err = err + (want.abs() + r.abs()) * 2.0 ** -24
    U.assert_within(y.cpu()[:, at], want, U.half_step(x, want.abs() + err) + err, "m %d n %d k %d" % (m, n, k))


@pytest.mark.parametrize("m,n,k", [(1, 20011, 32768), (3, 16385, 32768), (1, 16384, 28672), (1, 80000, 25600)])
@pytest.mark.parametrize("zeros", [False, True])
def test_long_rows_and_many_weights(m, n, k, zeros):
    edges = [0, 1, 15, 16, 16383, n - 2, n - 1] + [i for i in (16384, 16385, 16399, 16400) if i < n] + list(range(7, n, n // 23))
    _run(m, n, k, 128, F32, zeros, edges)


@pytest.mark.parametrize("m,n,k,group,x", [
    (32, 6144, 8192, 64, BF16),                             # an inbox beside more x than there is room for
    (300, 40000, 256, 64, BF16),                            # more tiles than an inbox holds
    (40, 3000, 8192, 128, F32)])
def test_many_rows(m, n, k, group, x):
    _run(m, n, k, group, x, True, range(3, n, n // 400))


@pytest.mark.parametrize("m", list(range(1, 20)) + [31, 33, 48])
@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("n,k,group", [(50, 1024, 32), (333, 4096, 64), (70, 640, 128)])
def test_every_number_of_rows(m, x, n, k, group):
    _run(m, n, k, group, x, True, seed=m)
