"""The host side of the bounded-cache calls without a GPU: which stream their
memory belongs to, what a step keeps between calls, and what is refused."""
import contextlib

import pytest
import torch

from paged_kv_cache_162_gb300 import engine as E


# ---------------------------------------------------------------- streams
class FakeStream:
    """Stands for a torch stream; remembers which streams it has waited for."""

    def __init__(self, handle):
        self.cuda_stream = handle
        self.waited = []

    def wait_stream(self, other):
        self.waited.append(other.cuda_stream)


class Streams:
    """Torch's streams as far as these calls use them, on the CPU: the handle
    of the current one, and on which each tensor was made or copied."""

    def __init__(self, monkeypatch):
        self.now = FakeStream(0)
        self.made = []
        monkeypatch.setattr(torch.cuda, "stream", self.on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
        for name in ("empty", "zeros", "full", "empty_like"):
            monkeypatch.setattr(torch, name, self.logged(name, getattr(torch, name)))
        for name in ("clone", "to", "copy_"):
            monkeypatch.setattr(torch.Tensor, name, self.logged(name, getattr(torch.Tensor, name)))

    def logged(self, name, real):
        def call(*args, **kw):
            self.made.append((name, self.now.cuda_stream))
            return real(*args, **kw)
        return call

    @contextlib.contextmanager
    def on(self, stream):
        before, self.now = self.now, stream
        yield
        self.now = before


@pytest.mark.parametrize("given", [77, FakeStream(77)])
def test_a_call_s_workspace_comes_from_its_own_stream(monkeypatch, given):
    """Memory that the current stream has given back may still be in use
    there: it must not become the scratch of a call on another stream."""
    streams = Streams(monkeypatch)
    E._workspace("call", 1024, torch.device("cpu"), given)
    assert streams.made == [("empty", 77)]
    E._workspace("call", 1024, torch.device("cpu"))
    assert streams.made[1:] == [("empty", 0)]
