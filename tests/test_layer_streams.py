"""Memory that the operators around the delta make for a call on a stream of
its own, host side (a stand-in for torch's allocator: no GPU)."""
import contextlib
import types

import heterogeneous_adapter_batching_amd.layer as layer


class Allocator:
    """Notes the stream that is current when a tensor is made, and the streams
    a tensor is recorded on."""

    def __init__(self):
        self.current = "the caller's"
        self.made = []
        self.cuda = types.SimpleNamespace(stream=self.stream, current_stream=lambda *a: self.current)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before

    def empty(self, shape, dtype=None, device=None):
        t = types.SimpleNamespace(pool=self.current, uses=[])
        t.record_stream = t.uses.append
        self.made.append(t)
        return t


def test_memory_comes_from_the_launch_stream(monkeypatch):
    """Memory handed out on a stream may still be in use by work queued there
    when its last owner let go of it: a launch on another stream would write
    under that work.  So it comes from the launch's own stream, and goes back
    only when the caller's stream is past its uses."""
    fake = Allocator()
    monkeypatch.setattr(layer, "torch", fake)
    t = layer._new((4, 8), "bf16", "cuda:0", "side")
    assert t.pool == "side" and t.uses == ["the caller's"]
    assert fake.current == "the caller's"


def test_no_stream_takes_the_current_one(monkeypatch):
    fake = Allocator()
    monkeypatch.setattr(layer, "torch", fake)
    t = layer._new((4, 8), "bf16", "cuda:0", None)
    assert t.pool == "the caller's" and t.uses == []
