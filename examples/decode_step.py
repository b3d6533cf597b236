"""One decode step around the experts, as a serving loop would run it: router ->
experts -> residual -> vocabulary projection -> next token, captured in a CUDA
graph and replayed.

    python examples/decode_step.py                      # 4-bit experts, one token
    python examples/decode_step.py --tokens 64 --weights bf16 --ranks 4
    python examples/decode_step.py --tokens 24 --norm --groups 8 --adapters 32 --vocab 50024

Weights are random.  With --ranks R the experts are R logical partitions, whose
partial results are added in rank order.  --norm puts an RMS norm in front of the
router and the experts, and one behind them; --groups G has the router choose among
the best half of G groups of experts; --adapters L adds one of L low-rank adapters (or
none) to each token's vocabulary projection (a vocabulary of a multiple of 8).
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import combine_send_counts_gb300 as ep  # noqa: E402


def random_weights(lead, N, K, group, gen):
    """[*lead, N, K] bf16, or its 4-bit form with zero points where group is not 0."""
    def one(*shape):
        return (torch.randn(shape, generator=gen, device="cuda") * K ** -0.5).to(torch.bfloat16)
    if group == 0:
        return one(*lead, N, K)
    if not lead:
        return ep.w4_quantize(one(N, K), group, zeros=True)
    parts = [ep.w4_quantize(one(N, K), group, zeros=True) for _ in range(lead[0])]   # never all of them in bf16
    return ep.W4(torch.stack([p.q for p in parts]), torch.stack([p.scale for p in parts]),
                 torch.stack([p.zero for p in parts]), group)


class DecodeStep:
    """The step with its weights and workspaces; group 0: bf16 experts."""

    def __init__(self, *, tokens, hidden, inter, experts, topk, vocab, group=128, head_group=128, ranks=1, seed=0,
                 norm=False, expert_groups=1, adapters=0, rank_of_adapters=16):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        local = experts // ranks
        self.wr = (torch.randn((experts, hidden), generator=gen, device="cuda") * hidden ** -0.5).to(torch.bfloat16)
        self.bias = torch.randn((experts,), generator=gen, device="cuda") * 0.01
        self.router = ep.RouterTopk(self.wr, topk, scoring="sigmoid", bias=self.bias, max_tokens=tokens,
                                    num_groups=expert_groups, topk_groups=(expert_groups + 1) // 2, group_score="top2")
        self.experts = [ep.MoeDecode(random_weights((local,), 2 * inter, hidden, group, gen),
                                     random_weights((local,), hidden, inter, group, gen), topk=topk,
                                     num_experts=experts, rank=r, max_tokens=tokens, out_dtype=torch.float32)
                        for r in range(ranks)]
        self.head = random_weights((), vocab, hidden, head_group, gen)
        self.norms = None
        if norm:
            self.norms = [(1 + 0.1 * torch.randn((hidden,), generator=gen, device="cuda")).to(torch.bfloat16)
                          for _ in range(2)]
        self.adapters = self.ids = None
        if adapters:
            if vocab % 8:
                raise ValueError("adapters need a vocabulary of a multiple of 8")
            down = torch.randn((adapters, rank_of_adapters, hidden), generator=gen, device="cuda") * hidden ** -0.5
            up = torch.randn((adapters, vocab, rank_of_adapters), generator=gen, device="cuda") * 0.01
            self.adapters = ep.LoraAdapters(down.to(torch.bfloat16), up.to(torch.bfloat16), max_tokens=tokens,
                                            out_dtype=torch.float32)
            self.ids = torch.randint(-1, adapters, (tokens,), generator=gen, device="cuda")

    def __call__(self, x):
        """x [T,hidden] bf16 -> (next token ids [T], logits [T,vocab] fp32, y [T,hidden] bf16)."""
        n = x if self.norms is None else ep.add_rms_norm(x, self.norms[0])["y"]
        idx, weights = self.router(n)
        y = x.float()
        if self.norms is None:
            for layer in self.experts:
                y = y + layer(n, idx, weights)
            y = y.to(torch.bfloat16)
        else:   # the residual stays in 32 bits up to the last norm, which adds the experts' sum to it
            part = self.experts[0](n, idx, weights)
            for layer in self.experts[1:]:
                part = part + layer(n, idx, weights)
            y = ep.add_rms_norm(part.to(torch.bfloat16), self.norms[1], y)["y"]
        logits = ep.w4_matvec(y, self.head, out_dtype=torch.float32)
        if self.adapters is not None:
            logits = self.adapters(y, self.ids[:x.shape[0]], logits, out=logits)
        return logits.argmax(dim=1), logits, y

    def check(self):
        """Raises if a device error was recorded."""
        for layer in (*self.experts, *([] if self.adapters is None else [self.adapters])):
            ep.raise_device_error(layer.err, "DecodeStep")

    def capture(self, x):
        """A graph of the step on the buffer x: (graph, outputs)."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self(x)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = self(x)
        return graph, out


def main():
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in dict(tokens=1, hidden=2048, inter=1024, experts=64, topk=6, vocab=50021, group=128, ranks=1,
                            groups=1, adapters=0, steps=100).items():
        a.add_argument("--" + name, type=int, default=value)
    a.add_argument("--norm", action="store_true")
    a.add_argument("--weights", choices=("int4", "bf16"), default="int4")
    a = a.parse_args()
    step = DecodeStep(tokens=a.tokens, hidden=a.hidden, inter=a.inter, experts=a.experts, topk=a.topk, vocab=a.vocab,
                      group=a.group if a.weights == "int4" else 0, head_group=a.group, ranks=a.ranks, norm=a.norm,
                      expert_groups=a.groups, adapters=a.adapters)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    graph, (token, _, _) = step.capture(x)
    for _ in range(3):
        graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    step.check()
    print(f"{begin.elapsed_time(end) * 1e3 / a.steps:.1f} us a step, tokens {token.tolist()[:8]}")


if __name__ == "__main__":
    main()
