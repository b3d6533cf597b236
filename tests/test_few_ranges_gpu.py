"""Parts of the few-token operators' ranges: biases as small as the scores'
differences, routers of thousands of tokens, experts with narrow results."""
import pytest
import torch

import combine_send_counts_gb300 as ep
import _few as f

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("spread", [0.003, 0.05])
@pytest.mark.parametrize("T,E,K", [(1, 256, 8), (7, 64, 6), (200, 33, 4)])
def test_small_biases_are_added_to_the_scores(scoring, spread, T, E, K):
    g = f.gen(E)
    x, w = f.randn((T, 512), g), f.randn((E, 512), g, 512 ** -0.5)
    bias = torch.randn((E,), generator=g, device="cuda") * spread
    logits = torch.empty((T, E), device="cuda")
    idx, wts = ep.RouterTopk(w, K, scoring=scoring, bias=bias, renormalize=False, max_tokens=T)(x, logits=logits)
    l = logits.double()
    score = torch.softmax(l, 1) if scoring == "softmax" else torch.sigmoid(l)
    key = score + bias.double()
    # exp and the sum of E terms in fp32, then the key's own rounding
    off = 2.0 ** -24 * ((E / 32 + 40) * score + key.abs()) + 2.0 ** -126
    lo, hi = (key - off).gather(1, idx), (key + off).gather(1, idx)
    assert (hi[:, :-1] >= lo[:, 1:]).all()                                  # descending
    chosen = torch.zeros_like(key, dtype=torch.bool).scatter_(1, idx, True)
    assert (chosen.sum(1) == K).all()
    best_left = torch.where(chosen, float("-inf"), key - off).amax(1)
    assert (hi.amin(1) >= best_left).all()                                  # and none better is left
    want = score.gather(1, idx)                                             # the bias stays out of the weights
    assert ((wts.double() - want).abs() <= 2.0 ** -24 * (E / 32 + 40) * want + 2.0 ** -126).all()
    # the two orders that a key without one of its parts would give are others
    for part in (score, bias.double().expand_as(key)):
        assert T == 1 or (part.topk(K, dim=1).indices != idx).any()


@pytest.mark.parametrize("T,H,E,K", [(1025, 256, 64, 6), (4097, 136, 33, 4), (16384, 512, 256, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_routers_of_many_tokens(T, H, E, K, dtype):
    g = f.gen(T)
    x, w = f.randn((T, H), g), f.randn((E, H), g, H ** -0.5, dtype)
    logits = torch.empty((T, E), device="cuda")
    r = ep.RouterTopk(w, K, max_tokens=T)
    idx, wts = r(x, logits=logits)
    f.assert_close(logits, x.double() @ w.double().t(), f.SUM * (x.double().abs() @ w.double().abs().t()))
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(idx, order.indices[:, :K])
    want = torch.softmax(order.values[:, :K].double(), 1)
    assert ((wts.double() - want).abs() <= 2.0 ** -24 * (E / 32 + 40) * want).all()
    again = r(x)
    assert torch.equal(again[0], idx) and torch.equal(again[1], wts)


@pytest.mark.parametrize("H", [32, 256, 512, 1056])
@pytest.mark.parametrize("fmt", ["bf16", 32])
@pytest.mark.parametrize("T,E", [(1, 64), (16, 64), (128, 64), (128, 3)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_narrow_results(H, fmt, T, E, out):
    g = f.gen(H + T)
    I, K = 416, min(E, 6)
    if fmt == "bf16":
        w13, w2 = f.randn((E, 2 * I, H), g, H ** -0.5), f.randn((E, H, I), g, I ** -0.5)
    else:
        w13, w2 = f.w4_random((E,), 2 * I, H, fmt, True, g), f.w4_random((E,), H, I, fmt, True, g)
    x = f.randn((T, H), g)
    idx, wts = f.routes(T, E, K, g)
    layer = ep.MoeDecode(w13, w2, topk=K, max_tokens=T, out_dtype=out)
    got = layer(x, idx, wts)
    want, tol = f.moe64(x, idx, wts, w13, w2, planes=3)
    f.assert_close(got, want, tol)
    assert torch.equal(got, layer(x, idx, wts))
