"""Kernels that start before the kernel ahead of them ends read what it wrote
through the ordinary path only: the read-only one is for memory that nobody
writes while the reader lives, and its loads may be moved ahead of the wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_send_counts_gb300", "csrc")
READ_ONLY = re.compile(r"__ldg\s*\(|\.nc\b|\bld_stream\s*\(|__restrict__")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", " ", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", " ", text)


FILES = sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh"))
               and (n == "ep_skinny.cuh" or '#include "ep_launch.cuh"' in code(n)))


def test_the_files_are_found():
    assert {"ep_moe.cuh", "ep_router.cu", "ep_skinny.cuh", "ep_w4.cu"} <= set(FILES)


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads(name):
    assert not READ_ONLY.findall(code(name))


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
def test_a_chain_without_waits_gives_the_bits_of_one_with_them(group):
    # every step reads what the one before wrote, in buffers that all rounds share
    import torch

    import _few as f
    import combine_send_counts_gb300 as ep

    g = f.gen(group)
    T, H, I, E, K = 12, 256, 128, 16, 4
    rounds = [dict(x=f.randn((T, H), g), w13=f.randn((E * 2 * I, H), g, H ** -0.5), w2=f.randn((E * H, I), g, I ** -0.5),
                   wr=f.randn((E, H), g, H ** -0.5)) for _ in range(6)]
    ws_r = torch.empty(ep.ep_router_workspace_size(T, H, E), dtype=torch.uint8, device="cuda")
    ws_m = torch.empty(ep.ep_moe_workspace_size(T, K, H, I), dtype=torch.uint8, device="cuda")
    q13, s13, z13 = (torch.empty((E * 2 * I, n), dtype=t, device="cuda")
                     for n, t in ((H // 2, torch.uint8), (H // group, torch.bfloat16), (H // group, torch.uint8)))
    q2, s2, z2 = (torch.empty((E * H, n), dtype=t, device="cuda")
                  for n, t in ((I // 2, torch.uint8), (I // group, torch.bfloat16), (I // group, torch.uint8)))
    back = torch.empty((E * 2 * I, H), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((T, K), dtype=torch.int64, device="cuda")
    wts = torch.empty((T, K), device="cuda")
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    err = ep.error_word()
    m13 = ep.EPMatrix(q13.data_ptr(), s13.data_ptr(), z13.data_ptr(), ep.EP_W_INT4, group)
    m2 = ep.EPMatrix(q2.data_ptr(), s2.data_ptr(), z2.data_ptr(), ep.EP_W_INT4, group)

    def chain(r, out, wait):
        steps = [lambda: ep.ep_w4_quantize(r["w13"], E * 2 * I, H, group, q13, s13, z13),
                 lambda: ep.ep_w4_dequantize(q13, s13, z13, E * 2 * I, H, group, back, 0),
                 lambda: ep.ep_w4_quantize(back, E * 2 * I, H, group, q13, s13, z13),
                 lambda: ep.ep_w4_quantize(r["w2"], E * H, I, group, q2, s2, z2),
                 lambda: ep.ep_w4_matvec(r["x"], T, q13, s13, z13, H, H, group, y, 0),
                 lambda: ep.ep_router_topk(y, T, H, r["wr"], 0, E, None, K, 0, 1, 1.0, idx, wts, None, ws_r),
                 lambda: ep.ep_moe_decode(y, idx, wts, T, K, H, I, E, E, 0, m13, m2, out, 1, ws_m, err)]
        for s in steps:
            s()
            if wait:
                torch.cuda.synchronize()

    apart, together = ([torch.empty((T, H), device="cuda") for _ in rounds] for _ in range(2))
    for r, out in zip(rounds, apart):
        chain(r, out, True)
    torch.cuda.synchronize()
    for _ in range(5):
        for r, out in zip(rounds, together):
            chain(r, out, False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(apart, together))
    assert int(err.item()) == 0
