"""The operators around the routing on other streams, at once, and in graphs."""
import pytest
import torch

import _few as f
import combine_send_counts_gb300 as ep

pytestmark = pytest.mark.gpu

LONG = 500_000_000   # cycles: a quarter of a second


def norm(g, big):
    T, H = (3000, 2048) if big else (5, 512)
    x, res, w = f.randn((T, H), g), f.randn((T, H), g), f.randn((H,), g)
    return lambda **kw: tuple(ep.add_rms_norm(x, w, res, fp8=True, **kw)[k] for k in ("y", "residual", "q", "scale"))


def norm_backward(g, big):
    T, H = (3000, 2048) if big else (5, 512)
    dy, h, w, d = f.randn((T, H), g), f.randn((T, H), g), f.randn((H,), g), f.randn((T, H), g)
    return lambda **kw: tuple(ep.add_rms_norm_backward(dy, h, w, d, **kw)[k] for k in ("dx", "dweight"))


def select(g, big):
    l, b = f.randn((9000 if big else 5, 256), g, 1.0, torch.float32), f.randn((256,), g, 0.05, torch.float32)
    return lambda **kw: ep.router_select(l, 8, scoring="sigmoid", bias=b, num_groups=8, topk_groups=4, group_score="top2",
                                         **kw)


def select_backward(g, big):
    T = 9000 if big else 5
    l, d = f.randn((T, 256), g, 1.0, torch.float32), f.randn((T, 8), g, 1.0, torch.float32)
    idx, _ = f.routes(T, 256, 8, g)
    return lambda **kw: (ep.router_select_backward(l, idx, d, **kw),)


def router(g, big):
    x, w = f.randn((120 if big else 3, 1024), g), f.randn((64, 1024), g, 1 / 32)
    plan = ep.RouterTopk(w, 4, num_groups=8, topk_groups=2)
    return lambda **kw: plan(x, **kw)


def lora(g, big, R=16):
    M, K, N, L = (2500, 1024, 1024, 5) if big else (20, 512, 256, 5)
    a, b = f.randn((L, R, K), g, K ** -0.5), f.randn((L, N, R), g, R ** -0.5)
    x, y = f.randn((M, K), g), f.randn((M, N), g)
    ids = torch.randint(-1, L, (M // 50 + 1,), generator=g, device="cuda").repeat_interleave(50)[:M].contiguous()
    plan = ep.LoraAdapters(a, b, max_tokens=M)
    return lambda **kw: (plan(x, ids, y, **kw),)


def lora64(g, big):
    return lora(g, big, 64)


def lora128(g, big):
    return lora(g, big, 128)


KINDS = [norm, norm_backward, select, select_backward, router, lora, lora64, lora128]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("how", ["argument", "handle", "current"])
def test_on_another_stream(kind, big, how):
    call = kind(f.gen(1), big)
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG // 10)
        got = call() if how == "current" else None
    if how != "current":
        got = call(stream=side if how == "argument" else side.cuda_stream)
    side.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("big", [False, True])
def test_in_a_graph(kind, big):
    call = kind(f.gen(2), big)
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = call()
        second = call()   # the same scratch, one after the other
    for _ in range(3):
        for t in (*first, *second):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(first, want) and same(second, want)
    assert same(call(), want)


@pytest.mark.parametrize("one", [lora, lora64, lora128])
@pytest.mark.parametrize("other", [lora, lora64, lora128, norm_backward, select])
def test_two_streams_at_once(one, other):
    # blocks of both share the SMs, and the tensor memory
    calls = [one(f.gen(3), True), other(f.gen(4), True)]
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(LONG // 20)
    got = [[], []]
    for _ in range(10):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(c())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(v, want[i]) for v in got[i])


def test_scratch_is_not_handed_out_while_another_stream_uses_it():
    g = f.gen(5)
    a, b = f.randn((3, 16, 512), g), f.randn((3, 256, 16), g)
    x, ids = f.randn((20, 512), g), torch.randint(-1, 3, (20,), generator=g, device="cuda")
    make = lambda: ep.LoraAdapters(a, b, max_tokens=64)   # noqa: E731
    kept, want = make(), make()(x, ids)
    side = torch.cuda.Stream()
    make()(x, ids, stream=side)
    torch.cuda.synchronize()
    size, place = kept.ws.numel(), kept.ws.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    out = kept(x, ids, stream=side)
    del kept
    mine = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query()
    assert all(t.data_ptr() != place for t in mine)
    for t in mine:
        t.fill_(255)
    side.synchronize()
    assert torch.equal(out, want)


def test_made_after_the_streams_earlier_work():
    g = f.gen(6)
    a, b = f.randn((3, 16, 512), g), f.randn((3, 256, 16), g)
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    ep.LoraAdapters(a, b)
    assert torch.cuda.current_stream().query()


@pytest.mark.parametrize("big", [False, True])
def test_a_chain_without_waits_gives_the_bits_of_one_with_them(big):
    # every step reads what the one before wrote, in buffers that all rounds share
    g = f.gen(7)
    T, H, E, K, L, R = (1500 if big else 12), 512, 64, 4, 3, 16
    rounds = [dict(x=f.randn((T, H), g), w=f.randn((H,), g), wr=f.randn((E, H), g, H ** -0.5), a=f.randn((L, R, H), g, H ** -0.5),
                   b=f.randn((L, H, R), g)) for _ in range(5)]
    res, h, y, z = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    logits, dl = torch.empty((T, E), device="cuda"), torch.empty((T, E), device="cuda")
    idx, wts = torch.empty((T, K), dtype=torch.int64, device="cuda"), torch.empty((T, K), device="cuda")
    ids = torch.empty((T,), dtype=torch.int64, device="cuda")
    ws_r = torch.empty(ep.ep_router_workspace_size(T, H, E), dtype=torch.uint8, device="cuda")
    ws_l = torch.empty(ep.ep_lora_workspace_size(T, R), dtype=torch.uint8, device="cuda")
    ws_n = torch.empty(ep.ep_rms_norm_backward_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    ids.copy_(torch.arange(T, device="cuda") // 40 % (L + 1) - 1)

    def chain(q, out, wait):
        steps = [lambda: ep.ep_add_rms_norm(q["x"], res, 0, T, H, q["w"], 0, 1e-6, h, y, None, None, 0, 0),
                 lambda: ep.ep_router_topk_groups(y, T, H, q["wr"], 0, E, None, K, 1, 8, 4, 1, 1, 1.0, idx, wts, logits, ws_r),
                 lambda: ep.ep_router_select(logits, 0, T, E, None, K, 1, 8, 2, 0, 1, 1.0, idx, wts),
                 lambda: ep.ep_lora(y, T, H, ids, q["a"], q["b"], None, L, R, H, h, 0, z, 0, ws_l, None),
                 lambda: ep.ep_router_select_backward(logits, 0, T, E, idx, wts, K, 1, 0, 1.0, dl, None),
                 lambda: ep.ep_add_rms_norm_backward(z, h, y, 0, T, H, q["w"], 0, 1e-6, res, None, out[1], ws_n),
                 lambda: ep.ep_lora(res, T, H, ids, q["a"], q["b"], None, L, R, H, res, 0, res, 0, ws_l, None)]
        for s in steps:
            s()
            if wait:
                torch.cuda.synchronize()
        for to, t in zip(out, (res, None, dl, wts)):
            if t is not None:
                to.copy_(t)

    new = lambda: [(torch.empty_like(res), torch.empty(H, device="cuda"), torch.empty_like(dl), torch.empty_like(wts))  # noqa: E731
                   for _ in rounds]
    apart, together = new(), new()
    res.zero_()
    for q, out in zip(rounds, apart):
        chain(q, out, True)
    torch.cuda.synchronize()
    for _ in range(5):
        res.zero_()
        for q, out in zip(rounds, together):
            chain(q, out, False)
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(apart, together))


def listed(g, M, L, R=16):
    """Rows of many adapters, in lists; of 3000, half are one adapter's instead."""
    K, N = 512, 520
    a, b = f.randn((L, R, K), g, K ** -0.5), f.randn((L, N, R), g, R ** -0.5)
    x, y = f.randn((M, K), g), f.randn((M, N), g)
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda")
    if M == 3000:
        ids[:M // 2] = 3
    plan = ep.LoraAdapters(a, b, max_tokens=M)
    return lambda **kw: (plan(x, ids, y, **kw),)


@pytest.mark.parametrize("M,L", [(300, 40), (1500, 12), (3000, 40), (9000, 12)])
@pytest.mark.parametrize("other", [lora, lora64, lora128, None])
def test_lists_and_another_stream_at_once(M, L, other):
    calls = [listed(f.gen(5), M, L), listed(f.gen(6), 3000, 12, 64) if other is None else other(f.gen(7), True)]
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(LONG // 20)
    got = [[], []]
    for _ in range(10):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(c())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(v, want[i]) for v in got[i])


def test_one_workspace_for_a_chain_of_lists():
    # each call reads what the one before wrote, over the same list and parts, whose tiles are others each time
    g = f.gen(8)
    H, L, R = 512, 30, 16
    a, b = f.randn((L, R, H), g, H ** -0.5), f.randn((L, H, R), g, 0.1)
    x = f.randn((9000, H), g)
    plan = ep.LoraAdapters(a, b, max_tokens=9000)
    sizes = [1, 9000, 64, 65, 3000, 512, 700, 2049, 20, 8193, 100, 2048, 4096, 3]
    ids = []
    for i, M in enumerate(sizes):
        v = torch.randint(-1, L, (M,), generator=g, device="cuda")
        if i % 3 == 1:
            v = v[:M // 60 + 1].repeat_interleave(60)[:M].contiguous()
        elif i % 3 == 2:
            v[M // 3:] = L - 1
        ids.append(v)

    def run(wait):   # nothing but the plan's own kernels between two calls
        h, k = x.clone(), torch.empty_like(x)
        k.copy_(x)
        for v in ids * 2:
            m = v.shape[0]
            plan(h[:m], v, k[:m], out=k[:m])
            h, k = k, h
            if wait:
                torch.cuda.synchronize()
        return h, k

    want = run(True)
    for _ in range(5):
        assert same(run(False), want)
