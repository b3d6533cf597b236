"""Infinite and NaN hidden values and router weights: the logits against the
product's own definition, and the choice that follows from them."""
import pytest
import torch

import combine_send_counts_gb300 as ep

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def product(x, w):
    """x w^T in 64 bits, one product at a time: 0 * inf is NaN, inf - inf too."""
    return (x.double()[:, None, :] * w.double()[None]).sum(-1)


def check(x, w, scoring="softmax", K=3):
    T, E = x.shape[0], w.shape[0]
    logits = torch.empty((T, E), device="cuda")
    idx, wts = ep.RouterTopk(w, K, scoring=scoring, renormalize=False, max_tokens=T)(x, logits=logits)
    want = product(x, w)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(logits), torch.isnan(want))
    assert torch.equal(logits[~fin & ~torch.isnan(want)].double(), want[~fin & ~torch.isnan(want)])
    # 2^-17 of the absolute sum: eight steps of 2^-23, twice for the halves of 128 columns, and 64 additions of 2^-24
    x0, w0 = (torch.where(torch.isfinite(t), t, 0).double().abs() for t in (x, w))
    assert ((logits.double() - want).abs()[fin] <= (2.0 ** -17 * (x0 @ w0.t()))[fin]).all()
    key = torch.where(torch.isnan(want), -INF, want)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    assert torch.equal(idx, torch.where(order.values[:, :K] > -INF, order.indices[:, :K], -1))
    assert not torch.isnan(wts).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,H", [(9, 8), (20, 264)])
def test_values_of_x(dtype, scoring, T, H):
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g)
    w = torch.randn((40, H), generator=g).to(torch.bfloat16).to(dtype)   # fp32 weights of 8 bits: their later terms are 0
    # weights 1, 2, .. in column 5 and the like: distinct, with both signs and a 0
    w[:, 5] = torch.arange(-20, 20).to(dtype)
    for t, v in ((1, INF), (2, -INF), (3, NAN)):
        x[t, 5] = v
    x[4, [2, 6]] = INF
    x[5, 0], x[5, 7] = INF, -INF
    check(x.to(torch.bfloat16).cuda(), w.cuda(), scoring)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(9, 8), (20, 264)])
def test_values_of_weights(dtype, T, H):
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    w = torch.randn((40, H), generator=g).to(dtype)   # fp32 weights of 24 bits
    w[3, 1], w[17, 4], w[21, 7] = INF, -INF, NAN
    w[30, [0, 6]] = INF
    if dtype == torch.float32:
        w[33, 2] = torch.tensor(0x7f800001, dtype=torch.int32).view(torch.float32)   # a NaN by its lowest bit
        assert torch.isnan(w[33, 2])
    x[0, [1, 4]] = 0.0
    x[1, 1] = INF
    check(x.cuda(), w.cuda())
