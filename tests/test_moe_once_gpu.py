"""moe_decode: one call that waits for nothing, with the caller's error word."""
import pytest
import torch

import combine_send_counts_gb300 as ep
import _few as f

pytestmark = pytest.mark.gpu


def args(g):
    w13, w2 = f.randn((4, 64, 64), g, 0.125), f.randn((4, 64, 32), g, 0.2)
    return (f.randn((3, 64), g), *f.routes(3, 4, 2, g), w13, w2)


def test_does_not_wait():
    a = args(f.gen(1))
    ep.moe_decode(*a)
    torch.cuda.synchronize()
    torch.cuda._sleep(500_000_000)
    ep.moe_decode(*a)
    ep.moe_decode(*a, err=None, out_dtype=torch.float32)
    assert not torch.cuda.current_stream().query()


@pytest.mark.parametrize("bad", [4, -2])
def test_reports_to_the_callers_word(bad):
    x, idx, wts, w13, w2 = args(f.gen(2))
    idx[1, 0] = bad
    err = ep.error_word()
    got = ep.moe_decode(x, idx, wts, w13, w2, err=err, out_dtype=torch.float32)
    assert int(err.item()) == ep.EP_ERR_INVALID_EXPERT
    with pytest.raises(ep.EPError, match="INVALID_EXPERT"):
        ep.raise_device_error(err, "moe_decode")
    unseen = ep.moe_decode(x, idx, wts, w13, w2, out_dtype=torch.float32)   # ignored just the same
    idx[1, 0] = -1
    want, tol = f.moe64(x, idx, wts, w13, w2, planes=3)
    f.assert_close(got, want, tol)
    assert torch.equal(got, unseen)


def test_in_a_graph():
    a = args(f.gen(3))
    want = ep.moe_decode(*a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ep.moe_decode(*a)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
