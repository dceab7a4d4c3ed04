"""Biases of ``adjust_logits`` for many tokens, some of them several times: the same bits as additions one by one in fp32."""
import numpy as np
import pytest
import torch

from test_gpu_adjust_logits import _check, _inputs

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")


def one_by_one(x, ids, bias):
    """x plus the sum of its token's biases, those added up in their order from 0, all in fp32."""
    y = x.clone()
    for i in range(x.shape[0]):
        sums = {}
        for t, b in zip(ids[i].tolist(), bias[i].numpy()):
            if 0 <= t < x.shape[1]:
                sums[t] = np.float32(sums.get(t, np.float32(0)) + b)
        at = torch.tensor(list(sums), dtype=torch.long)
        y[i, at] = x[i, at] + torch.tensor(np.array(list(sums.values()), dtype=np.float32))
    return y


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("columns", [0, 17000])               # (words of 16 bits and of 32)
@pytest.mark.parametrize("n,v,biases,alike", [(2, 40000, 40000, 0), (3, 40000, 20000, 300), (1, 20011, 3000, 2999), (2, 300, 1000, 700), (5, 50000, 1, 0)])
def test_the_same_bits(n, v, biases, alike, columns, dtype):
    g = torch.Generator().manual_seed(biases)
    ids = torch.stack([torch.randperm(max(v, biases), generator=g)[:biases] for _ in range(n)]).int()
    ids[:, :alike] = torch.randint(-1, min(v, 40) + 1, (n, alike), generator=g).int()
    ids = torch.stack([r[torch.randperm(biases, generator=g)] for r in ids])
    ids[0, 0] = 2 ** 31 - 1
    ids[-1, -1] = -2 ** 31
    bias = torch.randn((n, biases), generator=g) * 5
    x = torch.randn((n, v), generator=g).to(dtype)
    kw = dict(tokens=torch.full((n, columns), 2 ** 31 - 1, dtype=torch.int32, device="cuda"), presence=torch.ones(n, device="cuda")) if columns else {}
    got = mk.adjust_logits(x.cuda(), bias_ids=ids.cuda(), bias=bias.cuda(), **kw)
    assert torch.equal(got.cpu(), one_by_one(x.float(), ids, bias).to(dtype))
    again = x.cuda()
    assert mk.adjust_logits(again, bias_ids=ids.cuda(), bias=bias.cuda(), out=again, **kw) is again and torch.equal(again, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v,columns,biases", [(3, 2000, 900, 1500), (2, 33000, 20000, 4000)])
def test_beside_a_history_and_a_mask(n, v, columns, biases, dtype):
    a, x = _inputs(n, v, columns, biases, seed=6)
    a["bias"] *= 0.01                                        # (the bound grows with their number)
    _check(x.to(dtype).cuda(), a)
