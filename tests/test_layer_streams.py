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
        t = types.SimpleNamespace(pool=self.current, uses=[], device=device)
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


def test_a_plans_workspace_comes_from_its_upload_stream(monkeypatch):
    """The upload writes the workspace at once, on the stream it is given."""
    import heterogeneous_adapter_batching_amd as hab
    pool = hab.Pool(1, [64], [64], r_max=8, slab_ptr=1 << 30, slab_bytes=1 << 20)
    plan = hab.Plan(pool, 4, [0, 4], [-1])
    fake = Allocator()
    fake.uint8 = "uint8"
    empty = fake.empty

    def sized(n, dtype=None, device=None):
        t = empty(n, dtype, device)
        t.data_ptr, t.numel, t.element_size = (lambda: 0), (lambda: n), (lambda: 1)
        return t

    fake.empty = sized
    sent = []
    plan.lib = types.SimpleNamespace(lora_plan_workspace_bytes=lambda *a: 512,
                                     lora_plan_upload=lambda h, ws, n, mp, s: sent.append(s) or 0,
                                     lora_plan_destroy=lambda h: 0)
    monkeypatch.setattr(hab.api, "_torch", lambda: fake)
    side = types.SimpleNamespace(cuda_stream=7)
    ws = plan.upload(1, stream=side).ws
    assert ws.pool is side and ws.uses == ["the caller's"] and sent == [7]
