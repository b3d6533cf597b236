"""Host-side refusals of the operators around the routing: every bad argument is
answered before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import _fake_device as fake
import combine_send_counts_gb300 as ep

P, BAD = 4096, 4104   # never dereferenced: an aligned address and one that is not 16-byte aligned
INVALID, UNSUPPORTED = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return ep.load()


def test_norm(lib):
    def f(x=P, r=P, rd=0, T=4, H=256, w=P, wd=0, eps=1e-6, s=P, y=P, q=None, sc=None, fmt=0, rnd=0):
        return lib.ep_add_rms_norm(x, r, rd, T, H, w, wd, eps, s, y, q, sc, fmt, rnd, None)

    for bad in (dict(T=-1), dict(H=0), dict(H=-8), dict(H=12), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None),
                dict(x=BAD), dict(r=BAD), dict(w=BAD), dict(s=BAD), dict(y=BAD), dict(s=None, y=None),
                dict(q=P), dict(q=BAD, sc=P), dict(q=P, sc=P + 2), dict(q=P, sc=P, fmt=3), dict(q=P, sc=P, fmt=-1),
                dict(q=P, sc=P, rnd=2)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(rd=2), dict(wd=2), dict(H=32776), dict(T=1 << 31), dict(q=P, sc=P, H=264),
                dict(q=P, sc=P, fmt=2, H=512), dict(q=P, sc=P, fmt=2, rnd=1, H=640)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(T=0, x=None) == ep.EP_OK


def test_norm_backward(lib):
    n = lib.ep_rms_norm_backward_workspace_size(4, 256)

    def f(g=P, h=P, r=P, rd=0, T=4, H=256, w=P, wd=0, eps=1e-6, dh=P, dx=P, dw=P, ws=P, size=n):
        return lib.ep_add_rms_norm_backward(g, h, r, rd, T, H, w, wd, eps, dh, dx, dw, ws, size, None)

    for bad in (dict(T=-1), dict(H=0), dict(H=12), dict(eps=-1.0), dict(g=None), dict(h=None), dict(g=BAD), dict(h=BAD),
                dict(r=BAD), dict(w=BAD), dict(dh=BAD), dict(dx=BAD), dict(dw=P + 2), dict(ws=None), dict(ws=P + 128),
                dict(size=n - 1), dict(dh=None, dx=None, dw=None)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(rd=2), dict(wd=2), dict(H=32776), dict(T=1 << 31)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(T=0, dw=None) == ep.EP_OK
    assert lib.ep_rms_norm_backward_workspace_size(-1, 8) == 0


def test_a_backward_workspace_serves_fewer_rows():
    for H in (8, 256, 1024, 2048, 4096, 7168, 8200, 16384, 32768):
        sizes = [ep.ep_rms_norm_backward_workspace_size(T, H) for T in (1, 5, 152, 153, 304, 1000, 5000, 100000)]
        assert sizes == sorted(sizes)


def test_select(lib):
    def f(l=P, dt=0, T=4, E=64, b=None, K=4, sc=0, g=8, kept=2, mark=0, norm=1, i=P, w=P):
        return lib.ep_router_select(l, dt, T, E, b, K, sc, g, kept, mark, norm, 1.0, i, w, None)

    for bad in (dict(T=-1), dict(E=0), dict(E=8193), dict(K=0), dict(K=33), dict(K=65), dict(E=8, g=1, kept=1, K=9),
                dict(sc=2), dict(g=0), dict(g=7), dict(kept=0), dict(kept=9), dict(mark=2), dict(l=None), dict(i=None),
                dict(w=None), dict(l=P + 2), dict(b=P + 2), dict(i=P + 4), dict(w=P + 2)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(dt=2), dict(T=1 << 31), dict(E=128, g=128, kept=2)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(T=0, l=None) == ep.EP_OK
    n = lib.ep_router_workspace_size(4, 64, 64)
    r = lambda g=8, kept=2, mark=0, ws=P, size=n, H=64: lib.ep_router_topk_groups(  # noqa: E731
        P, 4, H, P, 0, 64, None, 4, 0, g, kept, mark, 1, 1.0, P, P, None, ws, size, None)
    for bad in (dict(g=7), dict(kept=9), dict(mark=-1), dict(ws=None), dict(size=n - 1), dict(H=60), dict(g=1, ws=None)):
        assert r(**bad) == INVALID, bad


def test_select_backward(lib):
    def f(l=P, dt=0, T=4, E=64, i=P, g=P, K=4, sc=0, norm=1, o=2 * P, err=None):
        return lib.ep_router_select_backward(l, dt, T, E, i, g, K, sc, norm, 1.0, o, err, None)

    for bad in (dict(T=-1), dict(E=0), dict(E=8193), dict(K=0), dict(K=33), dict(sc=2), dict(l=None), dict(i=None),
                dict(g=None), dict(o=None), dict(o=P), dict(l=P + 2), dict(i=P + 4), dict(g=P + 2), dict(err=P + 2)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(dt=2), dict(T=1 << 31)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(T=0, l=None) == ep.EP_OK


def test_lora(lib):
    n = lib.ep_lora_workspace_size(4, 16)

    def f(x=P, M=4, K=64, i=P, a=P, b=P, s=None, L=2, R=16, N=64, base=P, bd=0, o=P, od=0, ws=P, size=n, err=None):
        return lib.ep_lora(x, M, K, i, a, b, s, L, R, N, base, bd, o, od, ws, size, err, None)

    for bad in (dict(M=-1), dict(K=0), dict(K=12), dict(N=0), dict(N=12), dict(R=0), dict(R=12), dict(L=0), dict(x=None),
                dict(i=None), dict(a=None), dict(b=None), dict(o=None), dict(x=BAD), dict(a=BAD), dict(b=BAD),
                dict(base=BAD), dict(o=BAD), dict(i=P + 4), dict(s=P + 2), dict(err=P + 2), dict(bd=1), dict(od=1),
                dict(ws=None), dict(ws=P + 128), dict(size=n - 1)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(od=2), dict(bd=2), dict(R=136), dict(K=(1 << 24) + 8), dict(N=(1 << 24) + 8), dict(M=(1 << 24) + 1)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(M=0, x=None) == ep.EP_OK
    assert lib.ep_lora_workspace_size(-1, 16) == 0


def test_a_lora_workspace_serves_fewer_rows():
    sizes = [ep.ep_lora_workspace_size(M, 64) for M in (1, 2, 100, 1024, 1025, 2000, 2432, 2433, 5000, 38912, 38913, 100000)]
    assert sizes == sorted(sizes)


# ------------------------------------------------------------------- python --
T, H, E, K = 3, 256, 16, 2


def on(*shape, dtype=torch.float32):
    return fake.on(*shape, dtype=dtype)


def bf(*shape):
    return fake.on(*shape)


@pytest.fixture
def recorded(monkeypatch):
    return fake.install(monkeypatch)[0]


@pytest.mark.parametrize("call,what", [
    (lambda: ep.add_rms_norm(on(T, H), bf(H)), TypeError),
    (lambda: ep.add_rms_norm(bf(T, H, 1), bf(H)), ValueError),
    (lambda: ep.add_rms_norm(bf(T, H), bf(H + 8)), ValueError),
    (lambda: ep.add_rms_norm(bf(T, H), on(H, dtype=torch.float16)), TypeError),
    (lambda: ep.add_rms_norm(bf(T, H), bf(H), on(T, H, dtype=torch.float16)), TypeError),
    (lambda: ep.add_rms_norm(bf(T, H), bf(H), bf(T, H + 8)), ValueError),
    (lambda: ep.add_rms_norm(bf(T, H), bf(H), y=False), ValueError),
    (lambda: ep.add_rms_norm(bf(T, H), bf(H), inplace=True), ValueError),
    (lambda: ep.add_rms_norm(bf(T, H), bf(H), fp8=True, scale_fmt=7), ValueError),
    (lambda: ep.add_rms_norm(bf(H, T).t(), bf(H)), ValueError),
    (lambda: ep.add_rms_norm(torch.zeros(T, H, dtype=torch.bfloat16), None), ValueError),
    (lambda: ep.add_rms_norm_backward(bf(T, H), bf(T, H), bf(H), on(T, H)), TypeError),
    (lambda: ep.add_rms_norm_backward(bf(T, H), bf(T, H + 8), bf(H)), ValueError),
    (lambda: ep.add_rms_norm_backward(on(T, H), bf(T, H), bf(H)), TypeError),
    (lambda: ep.router_select(on(T, E, dtype=torch.float16), K), TypeError),
    (lambda: ep.router_select(on(T, E), 0), ValueError),
    (lambda: ep.router_select(on(T, E), E + 1), ValueError),
    (lambda: ep.router_select(on(T, E), K, scoring="relu"), ValueError),
    (lambda: ep.router_select(on(T, E), K, num_groups=3), ValueError),
    (lambda: ep.router_select(on(T, E), K, num_groups=4, topk_groups=5), ValueError),
    (lambda: ep.router_select(on(T, E), K, group_score="sum"), ValueError),
    (lambda: ep.router_select(on(T, E), K, bias=bf(E)), TypeError),
    (lambda: ep.router_select(on(E, T).t(), K), ValueError),
    (lambda: ep.RouterTopk(bf(E, H), K, num_groups=3), ValueError),
    (lambda: ep.RouterTopk(bf(E, H), K, num_groups=4, topk_groups=0), ValueError),
    (lambda: ep.router_select_backward(on(T, E), on(T, K, dtype=torch.int32), on(T, K)), TypeError),
    (lambda: ep.router_select_backward(on(T, E), on(T, K, dtype=torch.int64), on(T, K + 1)), ValueError),
    (lambda: ep.LoraAdapters(bf(2, 16, H), bf(3, 64, 16)), ValueError),
    (lambda: ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 8)), ValueError),
    (lambda: ep.LoraAdapters(on(2, 16, H), bf(2, 64, 16)), TypeError),
    (lambda: ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 16), on(3)), ValueError),
    (lambda: ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 16), out_dtype=torch.float16), TypeError),
    (lambda: ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 16))(bf(T, H + 8), on(T, dtype=torch.int64)), ValueError),
    (lambda: ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 16))(bf(T, H), on(T, dtype=torch.int32)), TypeError),
    (lambda: ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 16))(bf(T, H), on(T, dtype=torch.int64), bf(T, 72)), ValueError),
    (lambda: ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 16), max_tokens=2)(bf(T, H), on(T, dtype=torch.int64)), ValueError),
    (lambda: ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 16))(bf(T, H), on(T, dtype=torch.int64), out=on(T, 64)), TypeError),
])
def test_python_refuses(recorded, call, what):
    with pytest.raises(what):
        call()
    assert not recorded.calls


def test_overlapping_memory_is_refused(recorded):
    x = bf(2 * T, H)
    with pytest.raises(ValueError, match="overlap"):
        ep.add_rms_norm(x[:T], bf(H), x[1:T + 1], inplace=True)
    plan = ep.LoraAdapters(bf(2, 16, H), bf(2, H, 16))
    ids = on(T, dtype=torch.int64)
    for other in (dict(base=x[:T], out=x[1:T + 1]), dict(base=None, out=x[:T])):
        with pytest.raises(ValueError, match="overlap"):
            plan(x[:T], ids, other["base"], out=other["out"])
    assert not recorded.calls


def test_fields_are_fixed():
    with pytest.MonkeyPatch.context() as m:
        fake.install(m)
        plan = ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 16))
        with pytest.raises(AttributeError):
            plan.a = bf(2, 16, H)
        with pytest.raises(TypeError):
            plan.__reduce_ex__(4)


CALLS = [lambda: ep.add_rms_norm(bf(T, H), bf(H), bf(T, H), fp8=True),
         lambda: ep.add_rms_norm_backward(bf(T, H), bf(T, H), bf(H)),
         lambda: ep.router_select(on(T, E), K),
         lambda: ep.router_select_backward(on(T, E), on(T, K, dtype=torch.int64), on(T, K)),
         lambda: ep.RouterTopk(bf(E, H), K, num_groups=4, topk_groups=2)(bf(T, H)),
         lambda: ep.LoraAdapters(bf(2, 16, H), bf(2, 64, 16))(bf(T, H), on(T, dtype=torch.int64), on(T, 64))]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_current_in_the_call(monkeypatch, call, current):
    lib, state = fake.install(monkeypatch, current)
    call()
    assert len(lib.calls) == 1
    name, device, args = lib.calls[0]
    assert device == 1, name
    assert 101 in args   # and the stream is that device's
    assert state["device"] == current


def test_structures_are_as_the_header_says():
    assert (ep.EP_GROUP_MAX, ep.EP_GROUP_TOP2) == (0, 1)
    assert ctypes.sizeof(ctypes.c_size_t) == 8
