"""The experts keep all 24 bits of h between their two products, whatever the
type of the result."""
import pytest
import torch

import combine_send_counts_gb300 as ep

pytestmark = pytest.mark.gpu


def int4_of(w, group, step):
    """4-bit weights of exactly these values: codes of `step` in each group."""
    s = torch.empty((*w.shape[:-1], w.shape[-1] // group))
    s[...] = step
    q = (w.view(*s.shape, group) / s[..., None] + 8).to(torch.uint8).view(w.shape)
    assert ((q.float() - 8).view(*s.shape, group) * s[..., None]).view(w.shape).equal(w)
    return ep.W4((q[..., 0::2] | q[..., 1::2] << 4).cuda(), s.to(torch.bfloat16).cuda(), None, group)


@pytest.mark.parametrize("fmt", ["bf16", 32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 16])
def test_bits_of_h(fmt, out, T):
    # gate = 64, whose silu is 64 in fp32; up = 1 + 2^-8 + 2^-17 in element 0 and 1 + 2^-8 in element 1.  The result is
    # their difference, 64 * 2^-17 = 2^-11.  Every product and sum is exact in fp32, so the bound is that of matrix
    # steps that may truncate: eight of 2^-23 of the absolute sum of 129.
    H = I = 96
    x = torch.zeros((T, H))
    x[:, [0, 32, 64]] = 1.0
    w13, w2 = torch.zeros((1, 2 * I, H)), torch.zeros((1, H, I))
    w13[0, [0, 1], 0] = 64.0
    w13[0, I, 0], w13[0, I, 32], w13[0, I, 64] = 1.0, 2.0 ** -8, 2.0 ** -17
    w13[0, I + 1, 0], w13[0, I + 1, 32] = 1.0, 2.0 ** -8
    w2[0, :, 0], w2[0, :, 1] = 1.0, -1.0
    if fmt == "bf16":
        a, b = w13.to(torch.bfloat16).cuda(), w2.to(torch.bfloat16).cuda()
    else:
        step = torch.ones((1, 2 * I, H // fmt))
        step[0, :I] = 16.0   # a code of 4
        step[0, I:, 1], step[0, I:, 2] = 2.0 ** -8, 2.0 ** -17
        a, b = int4_of(w13, fmt, step), int4_of(w2, fmt, torch.ones((1, H, I // fmt)))
    idx = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    y = ep.moe_decode(x.to(torch.bfloat16).cuda(), idx, torch.ones((T, 1), device="cuda"), a, b, out_dtype=out)
    off = (y.double() - 2.0 ** -11).abs()
    assert (off <= 8 * 2.0 ** -23 * 129 + (2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -23) * 2.0 ** -11).all()


def test_large_terms_that_cancel_take_no_bits_of_small_ones():
    # h = 2^20 in elements 0 and 123, which cancel, and 1 + 2^-8 + 2^-16 in element 64 between them.  The first bf16
    # terms are integers below 2^24, whose sum is exact; the others are summed apart from them, so the result is exact.
    H, I = 24, 128
    x = torch.zeros((1, H))
    x[0, [0, 8, 16]] = 1.0
    w13, w2 = torch.zeros((1, 2 * I, H)), torch.zeros((1, H, I))
    w13[0, [0, 64, 123], 0] = 64.0
    w13[0, [I, I + 123], 0] = 2.0 ** 14
    w13[0, I + 64, [0, 8, 16]] = torch.tensor([2.0 ** -6, 2.0 ** -14, 2.0 ** -22])
    w2[0, :, [0, 64]] = 1.0
    w2[0, :, 123] = -1.0
    y = ep.moe_decode(x.to(torch.bfloat16).cuda(), torch.zeros((1, 1), dtype=torch.int64, device="cuda"),
                      torch.ones((1, 1), device="cuda"), w13.to(torch.bfloat16).cuda(), w2.to(torch.bfloat16).cuda(),
                      out_dtype=torch.float32)
    assert (y == 1 + 2.0 ** -8 + 2.0 ** -16).all()
