"""The scratch memory of kept objects, made on one stream and used on another."""
import pytest
import torch

import combine_send_counts_gb300 as ep
import _few as f

pytestmark = pytest.mark.gpu

LONG = 500_000_000   # cycles: a quarter of a second


def router(g):
    w = f.randn((64, 512), g, 512 ** -0.5)
    x = f.randn((16, 512), g)
    return lambda: ep.RouterTopk(w, 4), (x,)


def experts(g):
    w13, w2 = f.randn((8, 256, 512), g, 512 ** -0.5), f.randn((8, 512, 128), g, 128 ** -0.5)
    x = f.randn((16, 512), g)
    return lambda: ep.MoeDecode(w13, w2, topk=2), (x, *f.routes(16, 8, 2, g))


@pytest.mark.parametrize("kind", [router, experts])
def test_made_after_the_streams_earlier_work(kind):
    # the memory may have been that of a tensor which earlier work of this stream still writes
    make, _ = kind(f.gen(1))
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    assert not torch.cuda.current_stream().query()
    make()
    assert torch.cuda.current_stream().query()


@pytest.mark.parametrize("kind", [router, experts])
@pytest.mark.parametrize("how", ["argument", "handle", "current"])
def test_memory_is_not_handed_out_while_another_stream_uses_it(kind, how):
    make, args = kind(f.gen(2))
    kept = make()
    side = torch.cuda.Stream()
    make()(*args, stream=side)   # memory for the results on that stream: getting it from the driver would wait below
    torch.cuda.synchronize()
    size, place = kept.ws.numel(), kept.ws.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
        if how == "current":
            out = kept(*args)
    if how != "current":
        out = kept(*args, stream=side if how == "argument" else side.cuda_stream)
    del kept
    mine = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query()
    assert all(t.data_ptr() != place for t in mine)
    for t in mine:
        t.fill_(255)
    side.synchronize()
    want = make()(*args)
    for a, b in zip(out if isinstance(out, tuple) else (out,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(a, b)


def test_the_functional_router_does_not_wait():
    g = f.gen(3)
    w, x = f.randn((64, 512), g), f.randn((16, 512), g)
    ep.router_topk(x, w, 4)
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    ep.router_topk(x, w, 4)
    assert not torch.cuda.current_stream().query()


@pytest.mark.parametrize("kind", [router, experts])
def test_one_object_eagerly_and_in_a_graph_on_other_streams(kind):
    make, args = kind(f.gen(4))
    kept = make()
    want = kept(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept(*args, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kept(*args)
    graph.replay()
    torch.cuda.synchronize()
    pairs = zip(out, want) if isinstance(out, tuple) else [(out, want)]
    assert all(torch.equal(a, b) for a, b in pairs)
    del kept, out, graph
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
