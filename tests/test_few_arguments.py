"""What the few-token objects check and keep fixed (on the host, with a recording
library)."""
import copy
import pickle

import pytest
import torch

import _fake_device as fake
import combine_send_counts_gb300 as ep
from test_few_devices import E, H, I, K, T, w4

experts_args = lambda: (fake.on(T, H), fake.on(T, K, dtype=torch.int64), fake.on(T, K, dtype=torch.float32))  # noqa: E731


def experts():
    return ep.MoeDecode(w4(E, N=2 * I, K=H), w4(E, N=H, K=I), topk=K)


@pytest.mark.parametrize("once", [False, True])
def test_the_error_word_is_checked(monkeypatch, once):
    lib, _ = fake.install(monkeypatch, 1)

    def call(err):
        if once:
            return ep.moe_decode(*experts_args(), fake.on(E, 2 * I, H), fake.on(E, H, I), err=err)
        return experts()(*experts_args(), err=err)

    for shape in ((1,), (), (3,)):
        call(fake.on(*shape, dtype=torch.int32))
    assert len(lib.calls) == 3
    with pytest.raises(TypeError, match="err must be torch.int32"):
        call(fake.on(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="err must hold"):
        call(fake.on(0, dtype=torch.int32))
    with pytest.raises(ValueError, match="err must be on device 1"):
        call(torch.zeros(1, dtype=torch.int32))
    assert len(lib.calls) == 3


def test_fields_are_fixed(monkeypatch):
    # a call takes its pointers from the constructor: a field set later would be ignored, or checked in its place
    fake.install(monkeypatch, 1)
    w = w4(N=8, K=64)
    router = ep.RouterTopk(fake.on(E, H), K, bias=fake.on(E, dtype=torch.float32))
    layer = experts()
    for kept, names in ((w, ("q", "scale", "zero", "group", "shape")),
                        (router, ("w", "bias", "topk", "scoring", "renormalize", "scale", "max_tokens", "ws")),
                        (layer, ("w13", "w2", "rank", "topk", "max_tokens", "out_dtype", "err", "ws"))):
        for name in names:
            was = getattr(kept, name)
            with pytest.raises(AttributeError, match="fixed"):
                setattr(kept, name, None)
            with pytest.raises(AttributeError, match="fixed"):
                delattr(kept, name)
            assert getattr(kept, name) is was
    router.name = "of layer 3"   # a caller's own
    assert router.name == "of layer 3"


def test_w4_pointers_are_those_of_its_tensors(monkeypatch):
    lib, _ = fake.install(monkeypatch, 1)
    w = w4(N=8, K=64)
    ep.w4_matvec(fake.on(T, 64), w)
    ep.w4_dequantize(w)
    for name, _, args in lib.calls:
        assert w.q.data_ptr() in args and w.scale.data_ptr() in args, name


@pytest.mark.parametrize("copied", [copy.deepcopy, copy.copy, lambda w: pickle.loads(pickle.dumps(w))])
def test_a_copy_of_w4_points_to_its_own_tensors(copied):
    w = ep.W4(torch.ones((8, 32), dtype=torch.uint8), torch.ones((8, 2), dtype=torch.bfloat16),
              torch.ones((8, 2), dtype=torch.uint8), 32)
    c = copied(w)
    m = c.matrix
    assert (m.data, m.scale, m.zero) == (c.q.data_ptr(), c.scale.data_ptr(), c.zero.data_ptr())
    assert c.shape == w.shape and c.group == 32 and torch.equal(c.q, w.q) and torch.equal(c.zero, w.zero)


@pytest.mark.parametrize("copied", [copy.deepcopy, copy.copy, pickle.dumps])
def test_objects_with_scratch_are_not_copied(monkeypatch, copied):
    fake.install(monkeypatch, 1)
    for kept in (ep.RouterTopk(fake.on(E, H), K), experts()):
        with pytest.raises(TypeError, match="make another"):
            copied(kept)
