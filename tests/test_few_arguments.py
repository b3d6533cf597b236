"""What the few-token objects check and keep fixed (on the host, with a recording
library)."""
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
