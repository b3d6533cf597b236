"""The operators around the routing together, as a layer runs them: a decode step
with norms, groups of experts and adapters, and a training step's forward and
backward passes with the dispatch in between."""
import pytest
import torch

import _around as r
import _few as f
import combine_send_counts_gb300 as ep
from test_decode_example_gpu import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,experts,topk,vocab,groups,ranks,adapters", [
    (1, 256, 16, 4, 1032, 4, 1, 3), (5, 192, 12, 3, 520, 3, 3, 2), (33, 128, 8, 2, 304, 2, 2, 40)])
def test_decode_step(tokens, hidden, experts, topk, vocab, groups, ranks, adapters):
    step = example().DecodeStep(tokens=tokens, hidden=hidden, inter=64, experts=experts, topk=topk, vocab=vocab, group=64,
                                head_group=64, ranks=ranks, norm=True, expert_groups=groups, adapters=adapters)
    x = f.randn((tokens, hidden), f.gen(1))
    token, logits, y = step(x)
    # each step against 64 bits of what it was given
    n = ep.add_rms_norm(x, step.norms[0])["y"]
    _, n64 = r.norm64(x, step.norms[0], None, 1e-6)
    r.inside(n, n64, r.ROW * n64.abs())
    idx, weights = step.router(n)
    l = torch.empty((tokens, experts), device="cuda")
    assert torch.equal(step.router(n, l)[0], idx)
    want, w64 = r.select64(l, topk, scoring="sigmoid", bias=step.bias, num_groups=groups, topk_groups=(groups + 1) // 2,
                           group_score="top2")
    assert torch.equal(idx, want)
    r.inside(weights, w64, r.weights_tol(l, w64))
    part = step.experts[0](n, idx, weights)
    for layer in step.experts[1:]:
        part = part + layer(n, idx, weights)
    _, y64 = r.norm64(part.to(torch.bfloat16), step.norms[1], x.float(), 1e-6)
    r.inside(y, y64, r.ROW * y64.abs())
    base = ep.w4_matvec(y, step.head, out_dtype=torch.float32)
    out, tol = r.lora64(y, step.ids, step.adapters.a, step.adapters.b, None, base)
    r.inside(logits, out, tol)
    assert torch.equal(token, logits.argmax(dim=1))
    step.check()

    buffer = x.flip(0).contiguous()
    graph, got = step.capture(buffer)
    buffer.copy_(x)
    graph.replay()
    assert torch.equal(got[0], token) and torch.equal(got[1], logits) and torch.equal(got[2], y)
    step.check()


@pytest.mark.parametrize("T,H,E,K,P", [(257, 512, 64, 4, 4), (2000, 1024, 128, 8, 8)])
def test_training_step(T, H, E, K, P):
    g = f.gen(T)
    x, res = f.randn((T, H), g), f.randn((T, H), g)
    w = (1 + 0.1 * torch.randn((H,), generator=g, device="cuda")).to(torch.bfloat16)
    wr = f.randn((E, H), g, H ** -0.5)
    fwd = ep.add_rms_norm(x, w, res, fp8=True)
    h, y = fwd["residual"], fwd["y"]
    logits = (y.double() @ wr.double().t()).float()
    kw = dict(scoring="softmax", renormalize=True, scale=1.5)
    idx, weights = ep.router_select(logits, K, num_groups=8, topk_groups=4, group_score="max", **kw)
    # the rows in 8 bits go where the dispatch sends them: codes and scales are moved as they are
    route = ep.route_nosync(idx, weights, num_ranks=P, num_local_experts=E // P)
    N = int(route["rank_offsets"].view(-1)[-1].item())
    where = route["send_token_idx"][:N].long()
    codes = ep.dispatch_rows(fwd["q"].view(torch.bfloat16), route["token_pos"], N)
    scales = ep.dispatch_rows(fwd["scale"].view(torch.bfloat16), route["token_pos"], N)
    assert torch.equal(codes.view(torch.uint8), fwd["q"][where])
    assert torch.equal(scales.view(torch.float32), fwd["scale"][where])
    dw = f.randn((T, K), g, 0.1, torch.float32)
    dl = ep.router_select_backward(logits, idx, dw, **kw)
    want, tol = r.select_backward64(logits, idx, dw, **kw)
    r.inside(dl, want, tol)
    dy = (dl.double() @ wr.double()).to(torch.bfloat16)
    dres = f.randn((T, H), g, 0.01)
    back = ep.add_rms_norm_backward(dy, h, w, dres)
    dh, htol, dwn, wtol = r.norm_backward64(dy, h, w, dres, 1e-6)
    r.inside(back["dx"], dh, htol)
    r.inside(back["dweight"], dwn, wtol)
