"""The few-token calls run on their tensors' device, whichever is current (on
the host, with a library that records the current device)."""
import pytest
import torch

import _fake_device as fake
import combine_send_counts_gb300 as ep

H, I, E, T, K = 64, 32, 4, 3, 2


def w4(*lead, N, K):
    return ep.W4(fake.on(*lead, N, K // 2, dtype=torch.uint8), fake.on(*lead, N, K // 32), None, 32)


def quantize():
    ep.w4_quantize(fake.on(8, 64), 32)


def dequantize():
    ep.w4_dequantize(w4(N=8, K=64))


def matvec():
    ep.w4_matvec(fake.on(T, 64), w4(N=8, K=64))


def router():
    ep.RouterTopk(fake.on(E, H), K)(fake.on(T, H))


def router_once():
    ep.router_topk(fake.on(T, H), fake.on(E, H), K)


def experts(**kw):
    ep.MoeDecode(w4(E, N=2 * I, K=H), w4(E, N=H, K=I), topk=K)(
        fake.on(T, H), fake.on(T, K, dtype=torch.int64), fake.on(T, K, dtype=torch.float32), **kw)


def experts_once():
    ep.moe_decode(fake.on(T, H), fake.on(T, K, dtype=torch.int64), fake.on(T, K, dtype=torch.float32),
                  fake.on(E, 2 * I, H), fake.on(E, H, I))


@pytest.mark.parametrize("call", [quantize, dequantize, matvec, router, router_once, experts, experts_once])
@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_current_in_the_call(monkeypatch, call, current):
    lib, state = fake.install(monkeypatch, current)
    call()
    assert len(lib.calls) == 1
    name, device, args = lib.calls[0]
    assert device == 1, name
    assert 101 in args   # and the stream is that device's
    assert state["device"] == current
