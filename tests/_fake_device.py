"""Stands in for CUDA devices on the host: tensors that say they are on one, and
a library that records how it is called."""
from __future__ import annotations

import contextlib

import torch

import combine_send_counts_gb300 as ep


class On(torch.Tensor):
    """A host tensor whose get_device() is 1."""
    def get_device(self):
        return 1

    @property
    def is_cuda(self):
        return True


def on(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(On)


class Stream:
    """A stream of the fake device."""
    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def synchronize(self):
        self.log.append(("synchronize", self.cuda_stream))


class Library:
    """Answers size questions as the real one and records every other call with the current device."""

    def __init__(self, state):
        self.state, self.calls, self.real = state, [], ep.load()

    def __getattr__(self, name):
        if name.endswith("_size"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, self.state["device"], args))
            return 0
        return call


def install(monkeypatch, current=0, capturing=False):
    """-> (library, state): device `current` is current, and each device's current stream has the handle 100 + device."""
    state = {"device": current, "log": []}
    lib = Library(state)

    @contextlib.contextmanager
    def device(index):
        was, state["device"] = state["device"], index if isinstance(index, int) else 1
        yield
        state["device"] = was

    @contextlib.contextmanager
    def stream(s):
        was = state["device"]
        if s is not None:
            state["device"] = 1
        yield
        state["device"] = was

    monkeypatch.setattr(ep, "load", lambda: lib)
    monkeypatch.setattr(ep, "_current_device", lambda: state["device"], raising=False)
    monkeypatch.setattr(ep, "_current_raw", lambda index: 100 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(101, state["log"]))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    return lib, state
