"""Calls whose tensors, pool, plan or stream are on different devices, host
side: refused before anything is enqueued (no GPU)."""
import types

import pytest

import heterogeneous_adapter_batching_amd as hab
import heterogeneous_adapter_batching_amd.layer as layer

torch = pytest.importorskip("torch")


def parts(monkeypatch):
    """x and w on the device `here`, and what a call of sgmv_linear takes."""
    monkeypatch.setattr(layer, "_matrix", lambda t, *a: (0, t.shape[1]))
    calls = []
    monkeypatch.setattr(layer, "_enqueue", lambda *a: calls.append(a))
    x, w = torch.empty(4, 64, dtype=torch.bfloat16), torch.empty(64, 64, dtype=torch.bfloat16)
    lib = types.SimpleNamespace(sgmv_linear=None, sgmv_linear_plan_workspace_bytes=lambda *a: 0)
    here, there = torch.empty(1), torch.empty(1, device="meta")
    make = lambda slab, ws: (types.SimpleNamespace(lib=lib, handle=0, slab=slab),  # noqa: E731
                             types.SimpleNamespace(handle=0, ws=ws))
    return x, w, here, there, make, calls


def test_pool_and_plan_on_the_tensors_device(monkeypatch):
    x, w, here, there, make, calls = parts(monkeypatch)
    for slab, ws in ((there, here), (here, there)):
        with pytest.raises(ValueError, match="is on meta, not on cpu"):
            hab.sgmv_linear(*make(slab, ws), 0, [0], [0], x, w, y=x)
    assert not calls
    for slab, ws in ((here, here), (None, None)):     # (a pool over an address, a plan uploaded in C)
        hab.sgmv_linear(*make(slab, ws), 0, [0], [0], x, w, y=x)
    assert len(calls) == 2


def test_stream_of_another_device(monkeypatch):
    calls = []
    zero, one = torch.device("cuda", 0), torch.device("cuda", 1)
    monkeypatch.setattr(layer.torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    stream = types.SimpleNamespace(device=one, cuda_stream=5)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        layer._enqueue(lambda *a: calls.append(a) or 0, (), zero, stream)
    assert not calls
    layer._enqueue(lambda *a: calls.append(a) or 0, (), zero, types.SimpleNamespace(device=zero, cuda_stream=5))
    assert calls == [(5,)]
