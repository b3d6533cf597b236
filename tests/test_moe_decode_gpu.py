"""The experts for a few tokens against 64-bit sums: sizes, formats, routings,
masks, non-finite inputs, streams, graphs and large offsets."""
import pytest
import torch

import combine_send_counts_gb300 as ep
import _few as f

pytestmark = pytest.mark.gpu


def weights(El, H, I, fmt, g, zeros=False):
    if fmt == "bf16":
        return f.randn((El, 2 * I, H), g, H ** -0.5), f.randn((El, H, I), g, I ** -0.5)
    return f.w4_random((El,), 2 * I, H, fmt, zeros, g), f.w4_random((El,), H, I, fmt, zeros, g)


def check(T, H, I, E, El, rank, K, fmt, how, out, seed=0, zeros=False):
    g = f.gen(seed)
    w13, w2 = weights(El, H, I, fmt, g, zeros)
    x = f.randn((T, H), g)
    idx, wts = f.routes(T, E, K, g, how)
    layer = ep.MoeDecode(w13, w2, topk=K, num_experts=E, rank=rank, max_tokens=T, out_dtype=out)
    got = layer(x, idx, wts)
    want, tol = f.moe64(x, idx, wts, w13, w2, rank, planes=2 if out == torch.bfloat16 else 3)
    f.assert_close(got, want, tol)
    assert int(layer.err.item()) == 0
    assert torch.equal(got, layer(x, idx, wts))   # the same bits again
    return got


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 64, 128])
@pytest.mark.parametrize("fmt", ["bf16", 32, 128])
def test_tokens(T, fmt):
    check(T, 256, 128, 16, 16, 0, 4, fmt, "distinct", torch.bfloat16, seed=T)


@pytest.mark.parametrize("H,I", [(8, 8), (16, 24), (72, 40), (264, 136), (520, 8), (8, 520), (1000, 328), (2056, 1000),
                                 (7168, 64), (64, 2048), (4104, 16)])
@pytest.mark.parametrize("T", [1, 5, 20])
def test_sizes_bf16(H, I, T):
    check(T, H, I, 6, 6, 0, 3, "bf16", "distinct", torch.bfloat16, seed=H + I)


@pytest.mark.parametrize("group,H,I", [(32, 32, 32), (32, 96, 160), (32, 4128, 224), (64, 64, 192), (64, 4160, 1472),
                                       (128, 128, 128), (128, 384, 640), (128, 7168, 128), (64, 2112, 64)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T", [1, 11])
def test_sizes_int4(group, H, I, zeros, T):
    check(T, H, I, 6, 6, 0, 3, group, "distinct", torch.float32, seed=H + I, zeros=zeros)


@pytest.mark.parametrize("how", ["distinct", "repeats", "one", "none", "masked"])
@pytest.mark.parametrize("fmt", ["bf16", 64])
@pytest.mark.parametrize("T,K", [(1, 1), (1, 8), (3, 8), (40, 6), (128, 8)])
def test_routings(how, fmt, T, K):
    check(T, 192, 128, 12, 12, 0, K, fmt, how, torch.bfloat16, seed=K)


@pytest.mark.parametrize("fmt,H,I", [("bf16", 520, 1000), (32, 544, 1024), (64, 576, 960), (128, 640, 1152)])
@pytest.mark.parametrize("T,how", [(20, "repeats"), (60, "repeats"), (60, "one"), (90, "distinct")])
def test_several_passes_over_divided_experts(fmt, H, I, T, how):
    check(T, H, I, 6, 6, 0, 4, fmt, how, torch.float32, seed=T)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["bf16", 32])
@pytest.mark.parametrize("rank", [0, 1, 3])
def test_ranks(out, fmt, rank):
    check(19, 320, 96, 32, 8, rank, 5, fmt, "masked", out, seed=rank)


@pytest.mark.parametrize("E", [1, 2, 300, 8192])
def test_expert_counts(E):
    check(6, 64, 32, E, E, 0, min(E, 4), "bf16", "repeats", torch.float32, seed=E)


def test_ranks_add_up_to_the_whole_layer():
    g = f.gen(3)
    E, El, T, H, I, K = 16, 4, 12, 256, 64, 4
    w13, w2 = weights(E, H, I, "bf16", g)
    x = f.randn((T, H), g)
    idx, wts = f.routes(T, E, K, g)
    whole = ep.moe_decode(x, idx, wts, w13, w2, out_dtype=torch.float32)
    parts = sum(ep.moe_decode(x, idx, wts, w13[r * El:(r + 1) * El].contiguous(), w2[r * El:(r + 1) * El].contiguous(),
                              num_experts=E, rank=r, out_dtype=torch.float32).double() for r in range(E // El))
    want, tol = f.moe64(x, idx, wts, w13, w2, planes=3)
    f.assert_close(whole, want, tol)
    f.assert_close(parts.float(), want, tol + 4 * 2.0 ** -24 * want.abs())


def test_empty_batch():
    g = f.gen(4)
    w13, w2 = weights(4, 64, 32, "bf16", g)
    out = ep.MoeDecode(w13, w2, topk=2)(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"),
                                        torch.empty((0, 2), dtype=torch.int64, device="cuda"),
                                        torch.empty((0, 2), device="cuda"))
    assert out.shape == (0, 64)


@pytest.mark.parametrize("bad", [4, -2, 2 ** 40, -2 ** 40])
def test_invalid_ids_are_skipped_and_reported(bad):
    g = f.gen(5)
    w13, w2 = weights(4, 64, 32, "bf16", g)
    x = f.randn((3, 64), g)
    idx, wts = f.routes(3, 4, 2, g)
    idx[1, 0] = bad
    layer = ep.MoeDecode(w13, w2, topk=2, out_dtype=torch.float32)
    got = layer(x, idx, wts)
    assert int(layer.err.item()) == ep.EP_ERR_INVALID_EXPERT
    idx[1, 0] = -1
    want, tol = f.moe64(x, idx, wts, w13, w2, planes=3)
    f.assert_close(got, want, tol)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("fmt", ["bf16", 32])
def test_non_finite_rows_stay_their_own(value, fmt):
    # a token whose row holds it gets it; every other token's bits are as without it
    g = f.gen(6)
    w13, w2 = weights(8, 128, 64, fmt, g)
    x = f.randn((20, 128), g)
    idx, wts = f.routes(20, 8, 3, g)
    layer = ep.MoeDecode(w13, w2, topk=3, out_dtype=torch.float32)
    clean = layer(x, idx, wts)
    x2 = x.clone()
    x2[7, 5] = value
    got = layer(x2, idx, wts)
    assert not torch.isfinite(got[7]).any()
    keep = torch.arange(20, device="cuda") != 7
    assert torch.equal(got[keep], clean[keep])


def test_weights_of_slots_elsewhere_are_not_used():
    g = f.gen(7)
    w13, w2 = weights(4, 64, 32, "bf16", g)
    x = f.randn((6, 64), g)
    idx, wts = f.routes(6, 8, 4, g, "masked")
    layer = ep.MoeDecode(w13, w2, topk=4, num_experts=8, rank=1)
    a = layer(x, idx, wts)
    elsewhere = (idx < 4) | (idx >= 8)
    b = layer(x, idx, wts.masked_fill(elsewhere, float("nan")))
    assert torch.equal(a, b) and torch.isfinite(b.float()).all()
    assert (b[0] == 0).all()


def test_large_and_small_hidden_values():
    # silu overflows nothing, and products far from 1 keep their digits
    g = f.gen(8)
    w13, w2 = weights(2, 64, 32, "bf16", g)
    for scale in (2.0 ** 40, 2.0 ** -30):
        x = (f.randn((4, 64), g).float() * scale).to(torch.bfloat16)
        idx, wts = f.routes(4, 2, 2, g)
        got = ep.moe_decode(x, idx, wts, w13, w2, out_dtype=torch.float32)
        want, tol = f.moe64(x, idx, wts, w13, w2, planes=3)
        f.assert_close(got, want, tol)


def test_another_stream():
    g = f.gen(9)
    w13, w2 = weights(8, 512, 256, "bf16", g)
    x = f.randn((16, 512), g)
    idx, wts = f.routes(16, 8, 2, g)
    layer = ep.MoeDecode(w13, w2, topk=2)
    want = layer(x, idx, wts)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    by_argument = layer(x, idx, wts, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        as_current = layer(x, idx, wts)
        functional = ep.moe_decode(x, idx, wts, w13, w2, stream=side)
    side.synchronize()
    for got in (by_argument, as_current, functional):
        assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["bf16", 128])
def test_graph_replays_on_new_inputs(fmt):
    # the routing is read on the device: a captured call follows it
    g = f.gen(10)
    w13, w2 = weights(16, 256, 128, fmt, g)
    x = f.randn((8, 256), g)
    idx, wts = f.routes(8, 16, 4, g)
    layer = ep.MoeDecode(w13, w2, topk=4)
    out = torch.empty((8, 256), dtype=torch.bfloat16, device="cuda")
    layer(x, idx, wts, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, idx, wts, out=out)
    for how in ("distinct", "masked", "one", "none"):
        x.copy_(f.randn((8, 256), g))
        i2, w_2 = f.routes(8, 16, 4, g, how)
        idx.copy_(i2)
        wts.copy_(w_2)
        graph.replay()
        torch.cuda.synchronize()
        want, tol = f.moe64(x, idx, wts, w13, w2)
        f.assert_close(out, want, tol)


def test_back_to_back_calls_share_the_workspace():
    # calls of one stream follow one another without overlap, whatever starts early
    g = f.gen(11)
    w13, w2 = weights(16, 1024, 512, "bf16", g)
    layer = ep.MoeDecode(w13, w2, topk=4)
    sets = []
    for _ in range(6):
        x = f.randn((16, 1024), g)
        sets.append((x, *f.routes(16, 16, 4, g)))
    alone = []
    for s in sets:
        alone.append(layer(*s))
        torch.cuda.synchronize()
    together = [layer(*s) for _ in range(5) for s in sets]
    torch.cuda.synchronize()
    for i, got in enumerate(together):
        assert torch.equal(got, alone[i % len(sets)])


@pytest.mark.parametrize("fmt", ["bf16", 128])
def test_offsets_past_32_bits(fmt):
    # the last expert's matrices start past 2^31 elements and 2^32 bytes
    g = f.gen(12)
    H, I = 7168, 2048
    El = 100 if fmt == "bf16" else 320
    a, b = weights(1, H, I, fmt, g)
    if fmt == "bf16":
        w13 = torch.zeros((El, 2 * I, H), dtype=torch.bfloat16, device="cuda")
        w2 = torch.zeros((El, H, I), dtype=torch.bfloat16, device="cuda")
        w13[El - 1], w2[El - 1] = a[0], b[0]
    else:
        stack = []
        for one in (a, b):
            parts = []
            for t in (one.q, one.scale):
                big = torch.zeros((El, *t.shape[1:]), dtype=t.dtype, device="cuda")
                big[El - 1] = t[0]
                parts.append(big)
            stack.append(ep.W4(parts[0], parts[1], None, fmt))
        w13, w2 = stack
    assert w13.shape.numel() > 2 ** 31
    x = f.randn((2, H), g)
    idx = torch.tensor([[El - 1, 0], [-1, El - 1]], device="cuda")
    wts = torch.rand((2, 2), generator=g, device="cuda")
    got = ep.moe_decode(x, idx, wts, w13, w2, out_dtype=torch.float32)
    want, tol = f.moe64(x, torch.where(idx == El - 1, 0, -1), wts, a, b, planes=3)
    if fmt != "bf16":   # expert 0's codes are 0 with scale 0: every product is 0
        assert torch.isfinite(got).all()
    f.assert_close(got, want, tol)


def test_a_decode_layer_end_to_end():
    # router -> experts, as a decode step runs them, quantised weights included
    g = f.gen(13)
    T, H, I, E, K = 5, 256, 128, 16, 4
    x, wr = f.randn((T, H), g), f.randn((E, H), g, H ** -0.5)
    w13, w2 = weights(E, H, I, "bf16", g)
    q13, q2 = ep.w4_quantize(w13, 64), ep.w4_quantize(w2, 64, zeros=True)
    idx, wts = ep.router_topk(x, wr, K)
    assert idx.shape == (T, K) and torch.allclose(wts.sum(1), torch.ones(T, device="cuda"), atol=K * 2.0 ** -23)
    got = ep.moe_decode(x, idx, wts, q13, q2)
    want, tol = f.moe64(x, idx, wts, q13, q2)
    f.assert_close(got, want, tol)
