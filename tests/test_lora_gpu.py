"""LoraAdapters against 64 bits."""
import pytest
import torch

import _around as r
import _few as f
import combine_send_counts_gb300 as ep

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, None: None}


def inputs(M, K, N, L, R, base, how, g):
    x, a, b = f.randn((M, K), g), f.randn((L, R, K), g, K ** -0.5), f.randn((L, N, R), g, R ** -0.5)
    s = torch.rand((L,), generator=g, device="cuda") + 0.5
    y = None if base is None else f.randn((M, N), g, 1.0, TYPES[base])
    if how == "random":
        ids = torch.randint(-1, L, (M,), generator=g, device="cuda")
    elif how == "one":
        ids = torch.full((M,), L - 1, device="cuda")
    elif how == "none":
        ids = torch.full((M,), -1, device="cuda")
    else:   # runs of 37 rows
        ids = torch.randint(-1, L, (M // 37 + 1,), generator=g, device="cuda").repeat_interleave(37)[:M].contiguous()
    return x, ids, a, b, s, y


SIZES = [(1, 8, 8, 1, 8), (1, 4096, 4096, 4, 16), (3, 264, 72, 5, 24), (24, 2048, 1000, 32, 16), (17, 1024, 264, 2, 64),
         (33, 520, 520, 3, 128), (64, 4104, 256, 40, 32), (257, 256, 512, 7, 8), (1000, 264, 136, 9, 40),
         (1024, 512, 256, 300, 16), (1025, 512, 264, 6, 16), (1100, 264, 520, 3, 128), (1500, 1032, 40, 11, 64),
         (2000, 136, 2048, 70, 8), (40, 72, 24, 5, 120), (1050, 64, 48, 2, 96), (1030, 8, 8, 2, 8), (1300, 200, 72, 3, 24),
         (1040, 72, 264, 5, 40), (1200, 64, 96, 4, 72), (1100, 1000, 40, 2, 120), (1153, 448, 1000, 9, 32)]


@pytest.mark.parametrize("M,K,N,L,R", SIZES)
@pytest.mark.parametrize("base,out", [(None, "bf16"), ("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"),
                                      ("fp32", "fp32")])
@pytest.mark.parametrize("how", ["random", "one", "runs"])
def test_lora(M, K, N, L, R, base, out, how):
    g = f.gen(M + K + N + R)
    x, ids, a, b, s, y = inputs(M, K, N, L, R, base, how, g)
    plan = ep.LoraAdapters(a, b, s, max_tokens=M + 3, out_dtype=TYPES[out])
    got = plan(x, ids, y)
    want, tol = r.lora64(x, ids, a, b, s, y)
    assert got.dtype == TYPES[out] and int(plan.err.item()) == 0
    r.inside(got, want, tol)
    assert torch.equal(plan(x, ids, y), got)
    if y is not None:
        off = ids < 0
        assert torch.equal(got[off], y[off].to(got.dtype))   # rows without an adapter keep their bits


@pytest.mark.parametrize("M", [5, 1100])
def test_in_place_and_no_scaling(M):
    g = f.gen(M)
    x, ids, a, b, _, y = inputs(M, 256, 512, 4, 16, "bf16", "random", g)
    plan = ep.LoraAdapters(a, b, max_tokens=M)
    want, tol = r.lora64(x, ids, a, b, None, y)
    got = plan(x, ids, y)
    r.inside(got, want, tol)
    mine = y.clone()
    assert plan(x, ids, mine, out=mine) is mine and torch.equal(mine, got)
    assert torch.equal(plan(x, torch.full_like(ids, -1), None), torch.zeros_like(got))
    both = torch.empty((2 * M, 512), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        plan(x, ids, both[:M], out=both[1:M + 1])


@pytest.mark.parametrize("M", [70, 1100])
def test_bad_ids_and_rows_of_their_own(M):
    g = f.gen(M + 1)
    x, ids, a, b, s, y = inputs(M, 256, 264, 4, 16, "bf16", "random", g)
    plan = ep.LoraAdapters(a, b, s, max_tokens=M)
    want = plan(x, ids, y)
    bad = ids.clone()
    bad[3], bad[60], bad[M - 1] = 4, -2, 1 << 40
    err = ep.error_word()
    got = plan(x, bad, y, err=err)
    assert int(err.item()) == ep.EP_ERR_INVALID_EXPERT and int(plan.err.item()) == 0
    other = torch.ones(M, dtype=torch.bool, device="cuda")
    other[[3, 60, M - 1]] = False
    assert torch.equal(got[other], want[other]) and torch.equal(got[~other], y[~other])
    x2 = x.clone()
    x2[5], x2[6, 1] = float("nan"), float("inf")
    odd = plan(x2, ids, y)
    other = torch.ones(M, dtype=torch.bool, device="cuda")
    other[[5, 6]] = False
    assert torch.equal(odd[other], want[other])


@pytest.mark.parametrize("M", [40, 1200])
@pytest.mark.parametrize("R", [16, 64, 128])
def test_a_broken_adapter_harms_its_own_rows_alone(M, R):
    g = f.gen(R)
    x, ids, a, b, s, y = inputs(M, 264, 136, 5, R, "bf16", "random", g)
    want = ep.LoraAdapters(a, b, s, max_tokens=M)(x, ids, y)
    a2, b2 = a.clone(), b.clone()
    a2[1], b2[3, :, 2] = float("inf"), float("nan")
    got = ep.LoraAdapters(a2, b2, s, max_tokens=M)(x, ids, y)
    whole = (ids != 1) & (ids != 3)
    assert torch.equal(got[whole], want[whole])
    assert not bool(torch.isfinite(got[ids == 3]).any()) and not bool(torch.isfinite(got[ids == 1]).all())


def test_infinities():
    g = f.gen(8)
    x, _, a, b, s, y = inputs(4, 64, 64, 2, 16, "fp32", "random", g)
    ids = torch.tensor([0, 1, 0, -1], device="cuda")
    x[0, 3] = float("inf")
    got = ep.LoraAdapters(a, b, s, out_dtype=torch.float32)(x, ids, y)
    assert not bool(torch.isfinite(got[0]).any())
    want, tol = r.lora64(x[1:], ids[1:], a, b, s, y[1:])
    r.inside(got[1:], want, tol)


def test_adapters_past_32_bits():
    L, R, K, N = 1100, 128, 16384, 64   # a: 2.3e9 elements
    g = f.gen(4)
    a = torch.zeros((L, R, K), dtype=torch.bfloat16, device="cuda")
    b = f.randn((L, N, R), g, R ** -0.5)
    a[-1] = f.randn((R, K), g, K ** -0.5)
    x = f.randn((20, K), g)
    for M in (20, 1100):
        xs = x if M == 20 else x.repeat(55, 1)
        ids = torch.full((M,), L - 1, device="cuda")
        got = ep.LoraAdapters(a, b, max_tokens=M, out_dtype=torch.float32)(xs, ids)
        want, tol = r.lora64(xs, ids * 0, a[-1:], b[-1:], None, None)
        r.inside(got, want, tol)


def test_rows_past_32_bits():
    M, K, N = 300001, 7168, 16   # x: 2.15e9 elements
    g = f.gen(5)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-3:] = f.randn((3, K), g)
    a, b = f.randn((2, 16, K), g, K ** -0.5), f.randn((2, N, 16), g)
    ids = torch.ones(M, dtype=torch.int64, device="cuda")
    ids[-1] = 0
    got = ep.LoraAdapters(a, b, max_tokens=M, out_dtype=torch.float32)(x, ids)
    want, tol = r.lora64(x[-3:], ids[-3:], a, b, None, None)
    r.inside(got[-3:], want, tol)
    assert bool((got[:-3] == 0).all())


def test_smaller_batches_than_the_workspace_is_for():
    g = f.gen(6)
    x, ids, a, b, s, y = inputs(3000, 2048, 128, 3, 16, "bf16", "random", g)
    plan = ep.LoraAdapters(a, b, s, max_tokens=3000)
    for M in (1, 2, 100, 1023, 1024, 1025, 2047, 3000):
        got = plan(x[:M], ids[:M], y[:M])
        want, tol = r.lora64(x[:M], ids[:M], a, b, s, y[:M])
        r.inside(got, want, tol)
    assert plan(x[:0], ids[:0], y[:0]).shape == (0, 128)


@pytest.mark.parametrize("M,K,N,L,R", [(65, 72, 264, 40, 16), (130, 264, 40, 130, 24), (513, 64, 72, 9, 8),
                                       (700, 136, 264, 200, 64), (2048, 72, 40, 3000, 16), (2049, 264, 136, 20, 32),
                                       (2500, 64, 264, 9, 128), (8192, 72, 136, 70, 16), (8192, 64, 40, 9, 64),
                                       (8193, 64, 72, 24, 8), (20000, 40, 72, 30, 16), (768, 72, 40, 8, 16), (769, 72, 40, 8, 16)])
@pytest.mark.parametrize("base,out", [("bf16", "bf16"), ("fp32", "bf16")])
@pytest.mark.parametrize("how", ["both", "turns", "last"])
def test_long_requests_beside_short_ones(M, K, N, L, R, base, out, how):
    g = f.gen(M + K + N + R + L)
    x, ids, a, b, s, y = inputs(M, K, N, L, R, base, "random", g)
    if how == "both":       # one adapter for a stretch of rows, and another for the next
        ids[M // 8:M // 2] = L - 1
        ids[M // 2:M // 2 + 300] = 0
    elif how == "turns":    # eight adapters in turn, one more in some rows
        ids = torch.arange(M, device="cuda") % min(8, L)
        ids[::300] = L - 1
    else:                   # none but the last rows
        ids[:M - 5] = -1
    plan = ep.LoraAdapters(a, b, s, max_tokens=M, out_dtype=TYPES[out])
    got = plan(x, ids, y)
    want, tol = r.lora64(x, ids, a, b, s, y)
    assert int(plan.err.item()) == 0
    r.inside(got, want, tol)
    assert torch.equal(plan(x, ids, y), got)   # though a list's order is as it comes
    if base == out:
        assert torch.equal(plan(x, ids, y, out=y), got)


def test_a_graph_of_long_and_short_requests_with_other_ids():
    M, L = 3000, 40
    g = f.gen(5)
    x, ids, a, b, s, y = inputs(M, 264, 136, L, 16, "bf16", "random", g)
    plan = ep.LoraAdapters(a, b, s, max_tokens=M)
    runs = ids[:M // 100 + 1].repeat_interleave(100)[:M].contiguous()
    want = [plan(x, i, y).clone() for i in (ids, runs)]
    mine, out = ids.clone(), torch.empty_like(want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan(x, mine, y, out=out)
    for i, w in zip((ids, runs, ids), (want[0], want[1], want[0])):
        mine.copy_(i)
        graph.replay()
        assert torch.equal(out, w)
    bad = runs.clone()
    bad[2999] = L
    plan(x, bad, y)
    assert int(plan.err.item()) == ep.EP_ERR_INVALID_EXPERT
