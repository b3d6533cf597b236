"""router_select, its backward pass and the router with groups against 64 bits."""
import pytest
import torch

import _around as r
import _few as f
import combine_send_counts_gb300 as ep

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def check(logits, K, **kw):
    idx, w = ep.router_select(logits, K, **kw)
    want, w64 = r.select64(logits, K, **kw)
    assert idx.dtype == torch.int64 and w.dtype == torch.float32
    assert torch.equal(idx, want), f"{int((idx != want).any(1).sum())} of {idx.shape[0]} tokens"
    r.inside(w, w64, r.weights_tol(logits, w64))
    again = ep.router_select(logits, K, **kw)
    assert torch.equal(idx, again[0]) and torch.equal(w, again[1])
    return idx, w


SIZES = [(1, 8, 1, 1, 2), (3, 60, 1, 1, 6), (5, 64, 8, 3, 6), (2, 256, 8, 4, 8), (700, 256, 8, 4, 8), (33, 160, 8, 3, 6),
         (9, 512, 16, 5, 8), (4, 72, 3, 2, 9), (3, 2, 2, 1, 1), (4, 16, 16, 9, 1), (5, 16, 16, 16, 16), (3, 600, 5, 2, 4),
         (6, 384, 1, 1, 32), (3, 1000, 50, 7, 10), (2, 8192, 64, 8, 32), (130, 33, 1, 1, 33 - 1), (17, 1, 1, 1, 1),
         (40, 128, 64, 20, 12), (40, 96, 32, 5, 7), (40, 100, 4, 1, 25)]


@pytest.mark.parametrize("T,E,groups,kept,K", SIZES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("mark", ["max", "top2"])
def test_select(T, E, groups, kept, K, dtype, scoring, bias, mark):
    g = f.gen(T * 7 + E)
    logits = f.randn((T, E), g, 1.5, TYPES[dtype])
    b = f.randn((E,), g, 0.05, torch.float32) if bias else None
    for norm in (True, False):
        check(logits, K, scoring=scoring, bias=b, num_groups=groups, topk_groups=kept, group_score=mark,
              renormalize=norm, scale=2.5)


@pytest.mark.parametrize("E,groups", [(256, 8), (64, 1), (160, 8), (1000, 10)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", ["none", "zeros", "fine", "wide"])
@pytest.mark.parametrize("mark", ["max", "top2"])
def test_keys_that_are_near_or_equal(E, groups, scoring, bias, mark):
    # logits on a grid, so that many keys are equal, some moved by the last bits, so that many are nearly so
    g = f.gen(E)
    T = 300
    l = torch.randint(-3, 4, (T, E), generator=g, device="cuda").float() * 0.5
    move = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float() * 2.0 ** -23
    l[T // 3:] += (l * move)[T // 3:]
    l[2 * T // 3:] = l[2 * T // 3:] * 4 + 20 * (scoring == "sigmoid")   # scores that 32 bits take for 1
    b = {"none": None, "zeros": torch.zeros(E, device="cuda"),
         "fine": torch.randint(-3, 4, (E,), generator=g, device="cuda").float() * 2.0 ** -24,
         "wide": torch.randint(-3, 4, (E,), generator=g, device="cuda").float()}[bias]
    check(l, 6, scoring=scoring, bias=b, num_groups=groups, topk_groups=max(1, groups // 2), group_score=mark)


@pytest.mark.parametrize("E,groups", [(256, 8), (64, 1), (60, 4), (1000, 10)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("mark", ["max", "top2"])
def test_masks_and_non_finite(E, groups, scoring, bias, mark):
    g = f.gen(E + 1)
    T, inf = 64, float("inf")
    l = f.randn((T, E), g, 1.0, torch.float32)
    l[torch.rand((T, E), generator=g, device="cuda") < 0.4] = -inf
    l[1] = -inf                        # nothing is left
    l[2, :] = float("nan")
    l[3, ::2] = float("nan")
    l[4, 3] = inf
    l[5, [1, 5, 7]] = inf
    l[6] = torch.finfo(torch.float32).min
    l[7] = 0.0
    l[8, 3:] = -inf                    # fewer than K
    l[9] = l[9] * 1e30
    l[10, :] = -0.0
    l[10, 1::2] = 0.0
    b = None
    if bias:
        b = f.randn((E,), g, 1.0, torch.float32)
        b[0], b[2], b[9], b[E // 2:E // 2 + E // groups] = float("nan"), -inf, inf, -inf
    kw = dict(scoring=scoring, bias=b, num_groups=groups, topk_groups=max(1, groups // 2), group_score=mark, scale=0.5)
    for norm in (True, False):
        idx, w = ep.router_select(l, 8, renormalize=norm, **kw)
        want, w64 = r.select64(l, 8, renormalize=norm, **kw)
        assert torch.equal(idx, want), torch.nonzero((idx != want).any(1)).tolist()
        rows = torch.ones(T, dtype=torch.bool, device="cuda")
        rows[9] = False   # arguments past what the bound counts
        r.inside(w[rows], w64[rows], r.weights_tol(l[rows], w64[rows]))


@pytest.mark.parametrize("E,groups", [(64, 8), (1000, 8), (63, 7)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_fewer_experts_than_slots_and_unaligned_rows(E, groups, dtype):
    T, g = 9, f.gen(E)
    room = f.randn((T * E + 8,), g, 1.0, TYPES[dtype])
    bias = f.randn((E + 4,), g, 0.1, torch.float32)
    for at in (0, 1, 2, 3):   # starts at any element
        l, b = room[at:at + T * E].view(T, E), bias[at:at + E]
        for K in (4, min(32, E // groups + 5)):
            check(l, K, scoring="sigmoid", bias=b, num_groups=groups, topk_groups=1, group_score="top2")
            check(l, K, scoring="softmax", num_groups=groups, topk_groups=1, group_score="max", renormalize=False)
        idx, w = ep.router_select(l, 4)
        got = ep.router_select_backward(l, idx, w, renormalize=False)
        want, tol = r.select_backward64(l, idx, w, scoring="softmax", renormalize=False, scale=1.0)
        r.inside(got, want, tol)


def test_uniform_logits_and_no_tokens():
    l = torch.zeros((50, 256), device="cuda")
    idx, w = check(l, 8, scoring="sigmoid", bias=torch.zeros(256, device="cuda"), num_groups=8, topk_groups=4,
                   group_score="top2")
    assert idx.tolist() == [list(range(8))] * 50
    idx, w = ep.router_select(l[:0], 8)
    assert idx.shape == (0, 8) and w.shape == (0, 8)


@pytest.mark.parametrize("T,E,groups,kept,K", [(1, 256, 8, 4, 8), (24, 160, 8, 3, 6), (130, 64, 4, 2, 4)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("mark", ["max", "top2"])
def test_router_with_groups(T, E, groups, kept, K, scoring, bias, mark):
    g = f.gen(T + E)
    H = 1024
    x, wr = f.randn((T, H), g), f.randn((E, H), g, H ** -0.5)
    b = f.randn((E,), g, 0.05, torch.float32) if bias else None
    kw = dict(scoring=scoring, bias=b, num_groups=groups, topk_groups=kept, group_score=mark, scale=2.0)
    logits = torch.empty((T, E), device="cuda")
    router = ep.RouterTopk(wr, K, max_tokens=T, **kw)
    idx, w = router(x, logits)
    assert f.assert_close(logits, x.double() @ wr.double().t(), f.SUM * (x.double().abs() @ wr.double().abs().t())) is None
    want, w64 = r.select64(logits, K, **kw)   # of the logits as they are
    assert torch.equal(idx, want)
    r.inside(w, w64, r.weights_tol(logits, w64))
    once = ep.router_topk(x, wr, K, **kw)
    mine = ep.router_select(logits, K, **kw)
    for a in (once, mine):
        assert torch.equal(a[0], idx) and torch.equal(a[1], w)


def test_router_without_groups_is_as_it_was():
    g = f.gen(1)
    x, wr = f.randn((20, 512), g), f.randn((64, 512), g, 512 ** -0.5)
    a = ep.router_topk(x, wr, 4)
    ws = torch.empty(ep.ep_router_workspace_size(20, 512, 64), dtype=torch.uint8, device="cuda")
    idx, w = torch.empty((20, 4), dtype=torch.int64, device="cuda"), torch.empty((20, 4), device="cuda")
    ep.ep_router_topk_groups(x, 20, 512, wr, 0, 64, None, 4, 0, 1, 1, 0, 1, 1.0, idx, w, None, ws)
    assert torch.equal(a[0], idx) and torch.equal(a[1], w)


@pytest.mark.parametrize("T,E,K", [(1, 8, 2), (3, 60, 6), (200, 64, 6), (700, 256, 8), (5, 1000, 32), (2, 8192, 8),
                                   (17, 1, 1), (9, 33, 4)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("how", ["distinct", "masked", "repeats", "none"])
def test_backward(T, E, K, dtype, scoring, norm, how):
    g = f.gen(T * 3 + E)
    logits = f.randn((T, E), g, 1.5, TYPES[dtype])
    idx, _ = f.routes(T, E, K, g, how)
    dw = f.randn((T, K), g, 1.0, torch.float32)
    err = ep.error_word()
    got = ep.router_select_backward(logits, idx, dw, scoring=scoring, renormalize=norm, scale=1.5, err=err)
    want, tol = r.select_backward64(logits, idx, dw, scoring=scoring, renormalize=norm, scale=1.5)
    assert got.dtype == logits.dtype and int(err.item()) == 0
    r.inside(got, want, tol)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [False, True])
def test_backward_against_differences(scoring, norm):
    T, E, K, step = 20, 64, 4, 1e-6
    g = f.gen(11)
    logits = f.randn((T, E), g, 1.0, torch.float32)
    idx, _ = ep.router_select(logits, K, scoring=scoring, renormalize=norm)
    dw = f.randn((T, K), g, 1.0, torch.float32)
    got = ep.router_select_backward(logits, idx, dw, scoring=scoring, renormalize=norm, scale=2.0).double()
    along = torch.randn((T, E), generator=g, device="cuda", dtype=torch.float64)

    def value(l):
        c = r.scores64(l, scoring).gather(1, idx)
        return (2.0 * (c / c.sum(1, keepdim=True) if norm else c) * dw.double()).sum()

    slope = (value(logits.double() + step * along) - value(logits.double() - step * along)) / (2 * step)
    assert abs(slope - (got * along).sum()) <= 1e-5 * dw.double().abs().sum()


def test_backward_of_bad_ids_and_masked_logits():
    g = f.gen(2)
    logits = f.randn((6, 16), g, 1.0, torch.float32)
    dw = f.randn((6, 3), g, 1.0, torch.float32)
    idx = torch.tensor([[0, 1, 2], [3, -1, 5], [16, 1, 2], [-2, 4, 5], [1 << 40, 0, 3], [7, 8, 9]], device="cuda")
    logits[0, 5], logits[5, 8] = float("-inf"), float("nan")
    logits[3] = float("nan")   # the softmax of nothing
    good = idx.where((idx >= -1) & (idx < 16), torch.full_like(idx, -1))
    for scoring in ("softmax", "sigmoid"):
        for norm in (False, True):
            err = ep.error_word()
            got = ep.router_select_backward(logits, idx, dw, scoring=scoring, renormalize=norm, err=err)
            assert int(err.item()) == ep.EP_ERR_INVALID_EXPERT
            same = ep.router_select_backward(logits, good, dw, scoring=scoring, renormalize=norm)
            assert torch.equal(got, same)
            assert bool(torch.isfinite(got).all()) and got[0, 5] == 0 and got[5, 8] == 0
            assert bool((got[3] == 0).all())
            want, tol = r.select_backward64(logits[1:3], good[1:3], dw[1:3], scoring=scoring, renormalize=norm, scale=1.0)
            r.inside(got[1:3], want, tol)


def test_backward_of_small_shares():
    # scores that vanish in 32 bits, whose shares do not
    l = torch.tensor([[-100.0, -101.0, -300.0, 0.0], [-500.0, -499.0, -498.0, -490.0]], device="cuda")
    idx = torch.tensor([[0, 1], [1, 2]], device="cuda")
    dw = torch.tensor([[1.0, -2.0], [0.5, 3.0]], device="cuda")
    got = ep.router_select_backward(l, idx, dw, scoring="sigmoid", renormalize=True)
    want, _ = r.select_backward64(l, idx, dw, scoring="sigmoid", renormalize=True, scale=1.0)
    r.inside(got, want, 1e-5 * want.abs())
