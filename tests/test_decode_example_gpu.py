"""The decode-step example: router, experts and projection together against
64-bit sums, eagerly and as a replayed graph."""
import importlib.util
import os

import pytest
import torch

import _few as f

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decode_step.py")


def example():
    spec = importlib.util.spec_from_file_location("decode_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk,vocab,group,ranks", [
    (1, 256, 128, 16, 4, 1031, 128, 1), (5, 192, 64, 12, 3, 517, 64, 3), (33, 128, 96, 8, 2, 300, 0, 2)])
def test_step(tokens, hidden, inter, experts, topk, vocab, group, ranks):
    step = example().DecodeStep(tokens=tokens, hidden=hidden, inter=inter, experts=experts, topk=topk, vocab=vocab,
                                group=group, head_group=group or 32, ranks=ranks)
    x = f.randn((tokens, hidden), f.gen(1))
    token, logits, y = step(x)
    idx, weights = step.router(x)
    want = x.double()
    tol = torch.zeros_like(want)
    for r, layer in enumerate(step.experts):
        part, off = f.moe64(x, idx, weights, layer.w13, layer.w2, r, planes=3)
        want = want + part
        # the partial's own rounding and that of its addition, both fp32
        tol = tol + off + 2.0 ** -23 * part.abs() + 2.0 ** -23 * want.abs()
    f.assert_close(y, want, tol)
    head = f.values64(step.head)
    f.assert_close(logits, y.double() @ head.t(), f.SUM * (y.double().abs() @ head.abs().t()))
    assert torch.equal(token, logits.argmax(dim=1))
    step.check()

    buffer = torch.empty_like(x)
    buffer.copy_(x.flip(0))
    graph, out = step.capture(buffer)
    buffer.copy_(x)
    graph.replay()
    assert torch.equal(out[0], token) and torch.equal(out[1], logits) and torch.equal(out[2], y)
    step.check()
