"""``matvec_q4`` with x rows of elements of very different size: what an element
is worth does not depend on its neighbours."""
import pytest
import torch

import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32 = torch.bfloat16, torch.float32


def _check(y, x, w, what):
    xd = x.to(U.F64)
    want = xd @ w.t()
    # a block's products: 16 chained sums at most; a multiply-add a block of 32 codes; the warps' and terms' sums
    err = (xd.abs() @ w.abs().t()) * ((16 + x.shape[1] / 32 + 32) * 2.0 ** -23)
    U.assert_within(y, want, U.half_step(x.dtype, want.abs() + err) + err, what)


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 200, 512), (9, 50, 256), (24, 64, 4096)])
@pytest.mark.parametrize("ratio", [2.0 ** 20, 2.0 ** 35, 2.0 ** 60, -2.0 ** 100])
def test_an_outlier_of_no_weight(x, zeros, group, m, n, k, ratio):
    g = torch.Generator().manual_seed(1)
    code = torch.randint(0, 16, (n, k), generator=g, dtype=torch.int32)
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.int32) if zeros else torch.full((n, k // group), 8, dtype=torch.int32)
    at = 37
    code[:, at] = z[:, at // group]                         # the outlier's weight is zero in every row
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    scales = ((torch.rand((n, k // group), generator=g) + 0.2) * 0.01).to(BF16)
    zz = z.to(torch.uint8) if zeros else None
    xs = torch.randn((m, k), generator=g).to(x)
    xs[:, at] = ratio
    y = mk.matvec_q4(xs.cuda(), codes.cuda(), scales.cuda(), zeros=None if zz is None else zz.cuda())
    _check(y, xs, U.dequantize(codes, scales, zz), "ratio %g" % ratio)


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("m,k", [(1, 512), (5, 256), (40, 1024)])
def test_every_element_alone(x, m, k):
    # row n of the weights has one code that is not zero, that of element n: y[m][n] is x[m][n] times a small number
    g = torch.Generator().manual_seed(2)
    code = torch.full((k, k), 8, dtype=torch.int32)
    i = torch.arange(k)
    code[i, i] = torch.randint(0, 8, (k,), generator=g, dtype=torch.int32)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    scales = torch.full((k, k // 64), 0.0078125).to(BF16)
    xs = (torch.randn((m, k), generator=g) * 2.0 ** torch.randint(-60, 61, (m, k), generator=g)).to(x)
    y = mk.matvec_q4(xs.cuda(), codes.cuda(), scales.cuda())
    _check(y, xs, U.dequantize(codes, scales), "alone")
