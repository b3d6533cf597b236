"""4-bit weights: the quantiser against its definition in IEEE fp32 (numpy), the
values read back, and the product with a few rows against 64-bit sums."""
import numpy as np
import pytest
import torch

import combine_send_counts_gb300 as ep
import _few as f

pytestmark = pytest.mark.gpu


def bf16_rn(a):
    with np.errstate(all="ignore"):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def quantize_np(w, group, zeros):
    """The definition, one fp32 operation after the other."""
    v = w.float().cpu().numpy().reshape(w.shape[0], -1, group)
    fin = np.isfinite(v).all(-1)
    safe = np.where(np.isfinite(v), v, np.float32(0))
    with np.errstate(all="ignore"):
        lo = np.minimum(safe.min(-1), np.float32(0))
        hi = np.maximum(safe.max(-1), np.float32(0))
        wide = hi / np.float32(15) - lo / np.float32(15) if zeros else np.maximum(hi, -lo) / np.float32(7)
        scale = bf16_rn(np.where(fin, wide, np.float32(np.inf)))
        s = scale.float().numpy()
        ok = fin & (s > 0)
        z = np.where(ok, np.clip(np.rint(-lo / s), 0, 15), 0).astype(np.float32) if zeros else np.full_like(s, 8)
        r = np.where(ok[..., None], np.rint(safe / s[..., None]), 0).astype(np.float32)
        q = np.clip(r + z[..., None], 0, 15).astype(np.uint8).reshape(w.shape)
    return q[:, 0::2] | (q[:, 1::2] << 4), scale, z.astype(np.uint8)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N,k", [(1, 1), (3, 1), (17, 5), (130, 3), (1031, 17)])
def test_quantize_is_its_definition(group, zeros, N, k):
    g = f.gen(N + k)
    w = f.randn((N, k * group), g, 0.02)
    got = ep.w4_quantize(w, group, zeros=zeros)
    q, s, z = quantize_np(w, group, zeros)
    assert np.array_equal(got.q.cpu().numpy(), q)
    assert torch.equal(got.scale.cpu(), s)
    assert (got.zero is None) == (not zeros)
    if zeros:
        assert np.array_equal(got.zero.cpu().numpy(), z)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_special_groups(group, zeros):
    inf, nan, big, tiny = float("inf"), float("nan"), 3.3895e38, 2.0 ** -133
    rows = []
    for fill, at in [(0.0, []), (-0.0, []), (1.0, []), (-3.0, []), (0.5, [(3, inf)]), (0.5, [(0, -inf)]),
                     (0.25, [(group - 1, nan)]), (0.0, [(1, big), (2, -big)]), (0.0, [(5, tiny), (6, -tiny)]),
                     (2.0 ** -126, [(7, 2.0 ** -120)]), (nan, []), (-1.0, [(9, 15.0)]), (7.5, [(2, -7.5), (4, 2.5)])]:
        r = torch.full((group,), fill)
        for i, v in at:
            r[i] = v
        rows.append(r)
    w = torch.stack(rows).to(torch.bfloat16).cuda()
    got = ep.w4_quantize(w, group, zeros=zeros)
    q, s, z = quantize_np(w, group, zeros)
    assert torch.equal(got.scale.cpu(), s)
    assert np.array_equal(got.q.cpu().numpy(), q)
    if zeros:
        assert np.array_equal(got.zero.cpu().numpy(), z)
    back = ep.w4_dequantize(got, torch.float32)
    finite = torch.isfinite(w.float()).all(1)
    assert torch.isnan(back[~finite]).all() and not torch.isnan(back[finite]).any()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("lead", [(), (3,)])
def test_dequantize_reads_the_codes_back(group, zeros, lead):
    w = f.w4_random(lead, 37, 5 * group, group, zeros, f.gen(group))
    want = f.values64(w)
    assert torch.equal(ep.w4_dequantize(w, torch.float32).double(), want)   # 12 significant bits: exact
    assert torch.equal(ep.w4_dequantize(w), want.to(torch.bfloat16))


def test_quantization_error_is_half_a_step():
    g = f.gen(1)
    w = f.randn((64, 512), g)
    for zeros in (False, True):
        w4 = ep.w4_quantize(w, 64, zeros=zeros)
        off = (ep.w4_dequantize(w4, torch.float32) - w.float()).abs().view(64, -1, 64)
        # half a step inside the range; at its ends the bf16 scale may lie up to 2^-8 below the exact one, over
        # at most 15 steps, and the zero point's own rounding moves an end by another half step
        step = w4.scale.float()[..., None]
        assert (off <= step * (1.0 + 15 * 2.0 ** -8 if zeros else 0.5 + 8 * 2.0 ** -8)).all()


def check_matvec(M, N, K, group, zeros, out, seed=0):
    g = f.gen(seed)
    w = f.w4_random((), N, K, group, zeros, g)
    x = f.randn((M, K), g)
    got = ep.w4_matvec(x, w, out_dtype=out)
    v = f.values64(w)
    f.assert_close(got, x.double() @ v.t(), f.SUM * (x.double().abs() @ v.abs().t()))
    assert torch.equal(got, ep.w4_matvec(x, w, out_dtype=out))


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 24, 25, 32, 33, 64, 100])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_matvec_rows(M, out):
    check_matvec(M, 200, 384, 64, False, out, seed=M)


@pytest.mark.parametrize("N", [1, 2, 7, 8, 15, 16, 17, 33, 250, 1031])
@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (96, 32), (64, 64), (192, 64), (128, 128), (640, 128),
                                     (7168, 128), (4128, 32)])
@pytest.mark.parametrize("zeros", [False, True])
def test_matvec_sizes(N, K, group, zeros):
    check_matvec(3, N, K, group, zeros, torch.float32, seed=N + K)


@pytest.mark.parametrize("N,K", [(50021, 256), (2048, 2048), (128, 65536), (20000, 1024)])
@pytest.mark.parametrize("M", [1, 12])
def test_matvec_larger(N, K, M):
    check_matvec(M, N, K, 128, True, torch.bfloat16, seed=N)


def test_matvec_one_row_without_batch_dimension():
    g = f.gen(2)
    w = f.w4_random((), 40, 128, 32, False, g)
    x = f.randn((128,), g)
    assert torch.equal(ep.w4_matvec(x, w), ep.w4_matvec(x[None], w)[0])


def test_matvec_empty():
    w = f.w4_random((), 40, 128, 32, False, f.gen(3))
    assert ep.w4_matvec(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"), w).shape == (0, 40)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_matvec_non_finite_rows_stay_their_own(value):
    g = f.gen(4)
    w = f.w4_random((), 70, 256, 64, True, g)
    x = f.randn((11, 256), g)
    clean = ep.w4_matvec(x, w, out_dtype=torch.float32)
    x[4, 100] = value
    got = ep.w4_matvec(x, w, out_dtype=torch.float32)
    keep = torch.arange(11, device="cuda") != 4
    assert torch.equal(got[keep], clean[keep])
    moved = torch.nonzero(f.values64(w)[:, 100] != 0)[:, 0]   # where the code is not its zero point
    assert not torch.isfinite(got[4, moved]).any()


def test_matvec_unquantisable_group_reads_as_nan():
    g = f.gen(5)
    wt = f.randn((20, 128), g)
    wt[3, 40] = float("inf")
    y = ep.w4_matvec(f.randn((2, 128), g), ep.w4_quantize(wt, 32), out_dtype=torch.float32)
    assert torch.isnan(y[:, 3]).all() and torch.isfinite(y[:, torch.arange(20, device="cuda") != 3]).all()


def test_views_of_larger_buffers():
    # scale and zero need only their own type's alignment
    g = f.gen(6)
    w = f.w4_random((), 33, 96, 32, True, g)
    x = f.randn((5, 96), g)
    want = ep.w4_matvec(x, w)
    sb = torch.empty(33 * 3 + 1, dtype=torch.bfloat16, device="cuda")
    zb = torch.empty(33 * 3 + 3, dtype=torch.uint8, device="cuda")
    s, z = sb[1:].view(33, 3), zb[3:].view(33, 3)
    s.copy_(w.scale)
    z.copy_(w.zero)
    odd = ep.W4(w.q, s, z, 32)
    assert torch.equal(ep.w4_matvec(x, odd), want)
    assert torch.equal(ep.w4_dequantize(odd), ep.w4_dequantize(w))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("at,zero_at", [(0, 0), (1, 0), (0, 1), (2, 2), (3, 5), (4, 4), (8, 8)])
def test_scales_at_any_element(group, at, zero_at):
    """Rows of whole units, whose scales are loaded together where their start allows it."""
    g = f.gen(at + 10 * zero_at)
    w = f.w4_random((), 333, 1024, group, True, g)
    n = w.scale.numel()
    s = torch.full((n + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
    z = torch.full((n + 16,), 255, dtype=torch.uint8, device="cuda")
    s[at:at + n], z[zero_at:zero_at + n] = w.scale.flatten(), w.zero.flatten()
    moved = ep.W4(w.q, s[at:at + n].view(w.scale.shape), z[zero_at:zero_at + n].view(w.zero.shape), group)
    x = f.randn((5, 1024), g)
    got = ep.w4_matvec(x, moved, out_dtype=torch.float32)
    v = f.values64(w)
    f.assert_close(got, x.double() @ v.t(), f.SUM * (x.double().abs() @ v.abs().t()))
    assert torch.equal(got, ep.w4_matvec(x, w, out_dtype=torch.float32))
    assert torch.equal(ep.w4_dequantize(moved), ep.w4_dequantize(w))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [9, 24, 40, 70])
@pytest.mark.parametrize("N", [2500, 9731])
def test_matvec_passes_over_divided_rows(group, M, N):
    check_matvec(M, N, 512, group, True, torch.bfloat16, seed=M + N)


def test_offsets_past_32_bits():
    # codes past 2^31 bytes: the last rows against 64 bits, and the whole by one column of x
    N, K = 640_000, 7168
    g = f.gen(7)
    w = f.w4_random((), N, K, 128, False, g)
    assert w.q.numel() > 2 ** 31
    x = f.randn((1, K), g)
    got = ep.w4_matvec(x, w, out_dtype=torch.float32)
    tail = ep.W4(w.q[-64:].contiguous(), w.scale[-64:].contiguous(), None, 128)
    v = f.values64(tail)
    f.assert_close(got[:, -64:], x.double() @ v.t(), f.SUM * (x.double().abs() @ v.abs().t()))
    back = torch.empty((N, K), dtype=torch.bfloat16, device="cuda")   # 9 GB
    ep.ep_w4_dequantize(w.q, w.scale, None, N, K, 128, back, 0)
    assert torch.equal(back[-64:], v.to(torch.bfloat16))
    again = ep.w4_quantize(back, 128)
    assert torch.equal(ep.w4_dequantize(ep.W4(again.q[-64:].contiguous(), again.scale[-64:].contiguous(), None, 128),
                                        torch.float32),
                       ep.w4_dequantize(ep.w4_quantize(back[-64:].contiguous(), 128), torch.float32))


def test_another_stream_and_graph():
    g = f.gen(8)
    w = f.w4_random((), 300, 512, 128, False, g)
    x = f.randn((4, 512), g)
    want = ep.w4_matvec(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = ep.w4_matvec(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ep.w4_matvec(x, w)
    x.copy_(f.randn((4, 512), g))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ep.w4_matvec(x, w))
