"""The router: logits against 64-bit sums, and the selection and weights against
their definition on the logits that the call itself returns."""
import pytest
import torch

import combine_send_counts_gb300 as ep
import _few as f

pytestmark = pytest.mark.gpu


def select64(logits, bias, K, scoring, norm, scale):
    """The definition in 64 bits on given fp32 logits."""
    l = logits.double()
    l = torch.where(torch.isnan(l), float("-inf"), l)
    if scoring == "softmax":
        m = l.amax(1, keepdim=True)
        p = torch.where(l == m, 1.0, torch.exp(l - m))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    key = l if bias is None else p + bias.double()
    key = torch.where(torch.isnan(key) | torch.isnan(logits), float("-inf"), key)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    idx = order.indices[:, :K]
    ok = order.values[:, :K] > float("-inf")
    w = torch.where(ok, p.gather(1, idx), 0.0)
    if norm:
        t = w.sum(1, keepdim=True)
        w = torch.where(t > 0, w / t, 0.0)
    return torch.where(ok, idx, -1), w * scale


def check(T, H, E, K, scoring="softmax", bias=False, norm=True, scale=1.0, dtype=torch.bfloat16, seed=0):
    g = f.gen(seed)
    x = f.randn((T, H), g)
    w = f.randn((E, H), g, H ** -0.5, dtype)
    # biases far apart, so that no rounding of a score changes the order
    b = (torch.randperm(E, generator=g, device="cuda").float() * 4.0) if bias else None
    r = ep.RouterTopk(w, K, scoring=scoring, bias=b, renormalize=norm, scale=scale, max_tokens=max(T, 1))
    logits = torch.empty((T, E), device="cuda")
    idx, wts = r(x, logits=logits)
    f.assert_close(logits, x.double() @ w.double().t(), f.SUM * (x.double().abs() @ w.double().abs().t()))
    wi, ww = select64(logits, b, K, scoring, norm, scale)
    assert torch.equal(idx, wi)
    # exp and the sums of E and K terms in fp32: below 2^-24 * (E / 32 + 40) of each weight
    assert ((wts.double() - ww).abs() <= 2.0 ** -24 * (E / 32 + 40) * ww.abs() + 2.0 ** -126).all()
    i2, w2 = r(x)   # without the logits, again: the same bits
    assert torch.equal(i2, idx) and torch.equal(w2, wts)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 33, 130, 1000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tokens(T, dtype):
    check(T, 256, 64, 6, dtype=dtype, seed=T)


@pytest.mark.parametrize("E,K", [(1, 1), (2, 1), (2, 2), (7, 7), (8, 3), (17, 8), (60, 4), (256, 8), (300, 32),
                                 (1000, 10), (8192, 16)])
@pytest.mark.parametrize("T", [1, 13])
def test_experts(E, K, T):
    check(T, 136, E, K, seed=E + K)


@pytest.mark.parametrize("H", [8, 16, 24, 72, 264, 1000, 2048, 7168, 8200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_hidden_sizes(H, dtype):
    check(5, H, 33, 4, dtype=dtype, seed=H)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_options(scoring, bias, norm, scale):
    check(9, 512, 48, 6, scoring, bias, norm, scale)


def one_hot_logits(values):
    """x and w whose product is exactly the given [T,E] table of bf16 values."""
    T, E = values.shape
    H = max(8, (T + 7) // 8 * 8)
    x = torch.zeros((T, H), device="cuda")
    x[torch.arange(T), torch.arange(T)] = 1.0
    w = torch.zeros((E, H), device="cuda")
    w[:, :T] = values.t()
    return x.to(torch.bfloat16), w.to(torch.bfloat16)


def test_ties_go_to_the_lowest_expert():
    v = torch.zeros((4, 40), device="cuda")
    v[1, [5, 39, 20]] = 2.0
    v[2] = -1.0
    v[3, ::2] = 1.0
    idx, _ = ep.router_topk(*one_hot_logits(v), 4)
    assert idx.tolist() == [[0, 1, 2, 3], [5, 20, 39, 0], [0, 1, 2, 3], [0, 2, 4, 6]]


def test_a_bias_masks_experts_and_stays_out_of_the_weights():
    v = torch.arange(12, device="cuda", dtype=torch.float32).repeat(3, 1)
    x, w = one_hot_logits(v)
    bias = torch.full((12,), float("-inf"), device="cuda")
    bias[[2, 7]] = 0.0
    for scoring in ("softmax", "sigmoid"):
        idx, wts = ep.router_topk(x, w, 4, scoring=scoring, bias=bias)
        assert idx.tolist() == [[7, 2, -1, -1]] * 3
        assert (wts[:, 2:] == 0).all() and (wts[:, :2] > 0).all()
        assert torch.allclose(wts.sum(1), torch.ones(3, device="cuda"), atol=2.0 ** -22)
    bias.fill_(float("nan"))
    idx, wts = ep.router_topk(x, w, 4, bias=bias)
    assert (idx == -1).all() and (wts == 0).all()
    # and the framework takes such rows as unrouted
    assert int(ep.route_nosync(idx, wts, 2, 6)["send_counts"].sum()) == 0


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [False, True])
def test_non_finite_logits(scoring, norm):
    inf, nan = float("inf"), float("nan")
    w = torch.zeros((6, 8), device="cuda", dtype=torch.float32)
    w[:, 0] = torch.tensor([1.0, nan, inf, -inf, 2.0, inf])       # token 0's logits
    w[:, 1] = torch.tensor([nan, nan, nan, nan, nan, nan])
    w = torch.nan_to_num(w, nan=0.0, posinf=0.0, neginf=0.0)      # finite weights; x makes the values
    x = torch.zeros((5, 8), device="cuda")
    x[0, 0], x[1, 1], x[2, 0], x[3, 0] = 1.0, 1.0, inf, nan
    w[:, 0] = torch.tensor([1.0, -1.0, 3.0, 0.0, 2.0, -2.0])
    w[:, 1] = 0.5
    x[:, 2:] = 0.0
    r = ep.RouterTopk(w, 4, scoring=scoring, renormalize=norm)
    logits = torch.empty((5, 6), device="cuda")
    idx, wts = r(x.to(torch.bfloat16), logits=logits)
    wi, ww = select64(logits, None, 4, scoring, norm, 1.0)
    assert torch.equal(idx, wi)
    assert torch.allclose(wts.double(), ww, rtol=2.0 ** -18, atol=0)
    assert (idx[3] == -1).all() and (wts[3] == 0).all()           # a row of NaN goes nowhere


def test_empty_batch():
    idx, wts = ep.RouterTopk(f.randn((8, 16), f.gen(0)), 2)(torch.empty((0, 16), dtype=torch.bfloat16, device="cuda"))
    assert idx.shape == (0, 2) and wts.shape == (0, 2)


def test_another_stream_and_graph():
    g = f.gen(3)
    w = f.randn((64, 512), g, 512 ** -0.5)
    x = f.randn((16, 512), g)
    r = ep.RouterTopk(w, 4)
    want = r(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = r(x, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx, wts = r(x)
    x.copy_(f.randn((16, 512), g))
    graph.replay()
    torch.cuda.synchronize()
    want = r(x)
    assert torch.equal(idx, want[0]) and torch.equal(wts, want[1])


@pytest.mark.parametrize("E", [17, 64, 256, 1000])
def test_one_workspace_serves_every_smaller_batch(E):
    g = f.gen(4)
    w = f.randn((E, 2048), g, 2048 ** -0.5)
    r = ep.RouterTopk(w, 2, max_tokens=300)
    x = f.randn((300, 2048), g)
    for T in (1, 7, 8, 9, 16, 17, 31, 32, 33, 64, 100, 152, 153, 200, 299, 300):
        assert r(x[:T])[0].shape == (T, 2)
    sizes = [ep.ep_router_workspace_size(T, 2048, E) for T in range(1, 400)]
    assert sizes == sorted(sizes)
