"""add_rms_norm and its backward pass against 64 bits."""
import pytest
import torch

import _around as r
import _few as f
import combine_send_counts_gb300 as ep

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, None: None}


def inputs(T, H, residual, weight, seed=0):
    g = f.gen(seed + T * 100003 + H)
    x = f.randn((T, H), g)
    res = None if residual is None else f.randn((T, H), g, 2.0, TYPES[residual])
    w = None if weight is None else (1 + 0.3 * torch.randn((H,), generator=g, device="cuda")).to(TYPES[weight])
    return x, w, res


def check_codes(q, scale, y, fmt, power):
    T, H = y.shape
    if fmt == ep.EP_SCALE_COL_UE8M0:
        codes = scale.view(torch.uint8).view(H // 512, T, 4).permute(1, 0, 2).reshape(T, H // 128)
        s = torch.exp2(codes.double() - 127)
    else:
        s = (scale if fmt == ep.EP_SCALE_ROW_F32 else scale.t()).double()
    assert s.shape == (T, H // 128)
    want = y.view(T, -1, 128).abs().amax(2).clamp(min=1e-4) / 448
    if power:
        assert torch.equal(torch.exp2(torch.log2(s).round()), s)
        assert bool((s >= want * (1 - 2 * r.ROW)).all()) and bool((s < 2 * want * (1 + 2 * r.ROW)).all())
    else:
        r.inside(s.float(), want, 2 * r.ROW * want)
    v = q.view(torch.float8_e4m3fn).double().view(T, -1, 128) * s[..., None]
    y = y.view(T, -1, 128)
    # half a step of e4m3, which is 2^-10 of the scale for the smallest codes
    off = (v - y).abs() - ((2.0 ** -4 + 2 * r.ROW) * y.abs() + 2.0 ** -10 * s[..., None])
    assert bool((off <= 0).all()), off.max().item()


@pytest.mark.parametrize("T,H", [(1, 8), (3, 120), (2, 1000), (1, 1032), (5, 2048), (152, 7168), (153, 7168), (400, 8),
                                 (300, 1024), (300, 1032), (170, 4168), (160, 8192), (160, 8200), (3, 16384), (2, 32768)])
@pytest.mark.parametrize("residual", [None, "bf16", "fp32"])
@pytest.mark.parametrize("weight", [None, "bf16", "fp32"])
def test_norm(T, H, residual, weight):
    x, w, res = inputs(T, H, residual, weight)
    h, y = r.norm64(x, w, res, 1e-5)
    got = ep.add_rms_norm(x, w, res, eps=1e-5)
    assert got["q"] is None and got["scale"] is None
    r.inside(got["y"], y, r.ROW * y.abs())
    assert got["residual"] is None if res is None else torch.equal(got["residual"], h)


@pytest.mark.parametrize("T,H", [(1, 128), (2, 512), (1, 7168), (152, 7168), (154, 7168), (333, 1536), (170, 2560),
                                 (160, 16384), (1, 32768)])
@pytest.mark.parametrize("fmt", [ep.EP_SCALE_ROW_F32, ep.EP_SCALE_COL_F32, ep.EP_SCALE_COL_UE8M0])
@pytest.mark.parametrize("residual", [None, "bf16", "fp32"])
def test_eight_bits(T, H, fmt, residual):
    if fmt == ep.EP_SCALE_COL_UE8M0 and H % 512 != 0:
        with pytest.raises(ep.EPError):
            ep.add_rms_norm(*inputs(T, H, residual, "bf16"), fp8=True, scale_fmt=fmt, round_scale=True)
        return
    x, w, res = inputs(T, H, residual, "bf16")
    x[0] *= 2.0 ** -10   # small values next to large ones
    x[-1, ::3] = 0
    for power in ((True,) if fmt == ep.EP_SCALE_COL_UE8M0 else (False, True)):
        for wants_y in (True, False):
            got = ep.add_rms_norm(x, w, res, y=wants_y, fp8=True, scale_fmt=fmt, round_scale=power)
            h, y = r.norm64(x, w, res, 1e-6)
            check_codes(got["q"], got["scale"], y, fmt, power)
            if wants_y:
                r.inside(got["y"], y, r.ROW * y.abs())
            else:
                assert got["y"] is None
            if res is not None:
                assert torch.equal(got["residual"], h)


@pytest.mark.parametrize("T,H", [(1, 7168), (300, 2048)])
def test_codes_halfway_between_two(T, H):
    # h and w of few bits: their products are exact, and many stand exactly halfway between two codes
    g = f.gen(H)
    h = (torch.randint(-31, 32, (T, H), generator=g, device="cuda").float() / 32).to(torch.bfloat16)
    h[:, ::128] = 7.0 / 8   # the largest after w, so that values in units of the scale are whole 64ths of h w
    w = torch.ones(H, device="cuda").to(torch.bfloat16)
    w[::128] = 2.0
    got = ep.add_rms_norm(h, w, None, fp8=True)
    d = (h.double() * w.double()).view(T, -1, 128)
    want = (d * 448 / d.abs().amax(2, keepdim=True)).float().to(torch.float8_e4m3fn).view(T, H)
    assert torch.equal(got["q"].view(torch.float8_e4m3fn).float(), want.float())


@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", [(1, 2048), (160, 7168), (160, 10000)])
def test_in_place(residual, T, H):
    x, w, res = inputs(T, H, residual, "bf16")
    want = ep.add_rms_norm(x, w, res)
    mine = res.clone()
    got = ep.add_rms_norm(x, w, mine, inplace=True)
    assert got["residual"] is mine
    assert torch.equal(mine, want["residual"]) and torch.equal(got["y"], want["y"])
    # y over x, at the C entry
    h, y = torch.empty_like(res), x.clone()
    ep.ep_add_rms_norm(y, res, int(residual == "fp32"), T, H, w, 0, 1e-6, h, y, None, None, 0, 0)
    assert torch.equal(y, want["y"]) and torch.equal(h, want["residual"])


def test_the_sum_alone():
    x, w, res = inputs(5, 1000, "fp32", "bf16")
    got = ep.add_rms_norm(x, w, res, y=False)
    assert got["y"] is None and torch.equal(got["residual"], x.float() + res)


def test_rows_are_their_own():
    x, w, res = inputs(7, 1024, "bf16", "bf16")
    want = ep.add_rms_norm(x, w, res, fp8=True)
    x2 = x.clone()
    x2[2, 5], x2[4, 9] = float("nan"), float("inf")
    got = ep.add_rms_norm(x2, w, res, fp8=True)
    keep = [0, 1, 3, 5, 6]
    for k in ("y", "residual", "q", "scale"):
        assert torch.equal(got[k][keep], want[k][keep])
    assert bool(torch.isnan(got["y"][2]).all())
    assert bool(torch.isnan(got["y"][4, 9])) and bool((got["y"][4, :9] == 0).all())


def test_zero_rows_and_no_rows():
    x = torch.zeros((3, 512), dtype=torch.bfloat16, device="cuda")
    got = ep.add_rms_norm(x, None, x.clone(), fp8=True)
    assert bool((got["y"] == 0).all()) and bool((got["q"] == 0).all())
    assert torch.equal(got["scale"], torch.full((3, 4), 1e-4, device="cuda") / 448)
    none = ep.add_rms_norm(x[:0], None, x[:0].clone(), fp8=True)
    assert none["y"].shape == (0, 512) and none["scale"].shape == (0, 4)
    back = ep.add_rms_norm_backward(x[:0], x[:0].clone(), None)
    assert back["dx"].shape == (0, 512) and bool((back["dweight"] == 0).all())


def test_more_elements_than_32_bits_count():
    T, H = 300001, 7168
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    g = f.gen(5)
    x[-2:] = f.randn((2, H), g)
    got = ep.add_rms_norm(x, None, None, fp8=True)
    _, y = r.norm64(x[-2:], None, None, 1e-6)
    r.inside(got["y"][-2:], y, r.ROW * y.abs())
    check_codes(got["q"][-2:], got["scale"][-2:], y, ep.EP_SCALE_ROW_F32, False)
    assert bool((got["y"][:4] == 0).all())
    dy = got["y"]
    back = ep.add_rms_norm_backward(dy, x, None)
    dh, tol, dw, wtol = r.norm_backward64(dy[-2:], x[-2:], None, None, 1e-6)
    r.inside(back["dx"][-2:], dh, tol)
    r.inside(back["dweight"], dw, wtol)


@pytest.mark.parametrize("T,H", [(1, 8), (2, 1000), (5, 2048), (152, 7168), (305, 1024), (700, 1032), (333, 4168),
                                 (160, 8192), (400, 8200), (200, 16384), (160, 32768), (3, 32768), (4096, 256)])
@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("weight", [None, "bf16", "fp32"])
@pytest.mark.parametrize("way", [False, True])
def test_backward(T, H, residual, weight, way):
    _, w, h = inputs(T, H, residual, weight)
    g = f.gen(T + H)
    dy = f.randn((T, H), g, 0.1)
    dres = f.randn((T, H), g, 0.1, h.dtype) if way else None
    got = ep.add_rms_norm_backward(dy, h, w, dres, eps=1e-5)
    dh, tol, dw, wtol = r.norm_backward64(dy, h, w, dres, 1e-5)
    assert got["dresidual"].dtype == h.dtype and got["dweight"].dtype == torch.float32
    r.inside(got["dresidual"], dh, tol)
    r.inside(got["dx"], dh, tol)
    r.inside(got["dweight"], dw, wtol)
    again = ep.add_rms_norm_backward(dy, h, w, dres, eps=1e-5)
    assert all(torch.equal(got[k], again[k]) for k in got)
    less = ep.add_rms_norm_backward(dy, h, w, dres, eps=1e-5, dweight=False)
    assert less["dweight"] is None and torch.equal(less["dresidual"], got["dresidual"])


def test_backward_against_differences():
    T, H, step = 6, 512, 1e-6
    g = f.gen(3)
    h, w = f.randn((T, H), g, 1.0, torch.float32), f.randn((H,), g, 1.0, torch.float32)
    dy = f.randn((T, H), g)
    got = ep.add_rms_norm_backward(dy, h, w, None, eps=1e-3)
    along, wide = (torch.randn(s, generator=g, device="cuda", dtype=torch.float64) for s in ((T, H), (H,)))

    def value(dh, dw):
        d = h.double() + dh
        n = d * torch.rsqrt(d.square().mean(1, keepdim=True) + 1e-3) * (w.double() + dw)
        return (n * dy.double()).sum()

    for dh, dw, mine in ((along * step, 0, (got["dresidual"].double() * along).sum()),
                         (0, wide * step, (got["dweight"].double() * wide).sum())):
        slope = (value(dh, dw) - value(-dh, -dw)) / (2 * step)
        assert abs(slope - mine) <= 1e-5 * (dy.double().abs().sum())   # rounded entries, and the square of the step


def test_backward_in_place():
    T, H = 200, 2048
    _, w, h = inputs(T, H, "bf16", "bf16")
    g = f.gen(9)
    dy, dres = f.randn((T, H), g), f.randn((T, H), g)
    want = ep.add_rms_norm_backward(dy, h, w, dres)
    ws = torch.empty(ep.ep_rms_norm_backward_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    for over in ("dres", "dy"):
        a, b, dw = dy.clone(), dres.clone(), torch.empty(H, device="cuda")
        ep.ep_add_rms_norm_backward(a, h, b, 0, T, H, w, 0, 1e-6, b if over == "dres" else a, None, dw, ws)
        assert torch.equal(b if over == "dres" else a, want["dx"]) and torch.equal(dw, want["dweight"])


@pytest.mark.parametrize("T,H", [(153, 8), (161, 256), (1001, 264), (155, 504), (999, 512), (154, 520), (1000, 1024)])
@pytest.mark.parametrize("residual", [None, "bf16", "fp32"])
def test_many_short_rows(T, H, residual):
    test_norm(T, H, residual, "bf16")


@pytest.mark.parametrize("T,H", [(153, 128), (999, 384), (1001, 512), (161, 256), (1000, 640)])
@pytest.mark.parametrize("fmt", [ep.EP_SCALE_ROW_F32, ep.EP_SCALE_COL_F32, ep.EP_SCALE_COL_UE8M0])
@pytest.mark.parametrize("residual", [None, "fp32"])
def test_eight_bits_of_many_short_rows(T, H, fmt, residual):
    test_eight_bits(T, H, fmt, residual)
