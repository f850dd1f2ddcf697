"""A plan's workspace and staging outlive the work that reads them."""
import pytest
import torch

import heterogeneous_adapter_batching_amd as hab
from attention_reference import Batch
from test_gpu_attention import plan_of, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["attention", "rotary"])
def test_a_workspace_replaced_behind_a_call_on_another_stream(call):
    """Its memory is not given out while the call is queued.  (A plan that is
    destroyed waits.)"""
    b = Batch([1] * 4, [300, 20, 4000, 9], seed=1, page=64)
    want = run(b)
    side = torch.cuda.Stream()
    plan = plan_of(b).upload().upload()          # (both staging buffers are there)
    at, size = plan.ws.data_ptr(), plan.ws.nbytes
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(int(4e8))              # (a fifth of a second)
    if call == "attention":
        o = hab.paged_attention(plan, b.q, b.k, b.v, b.pages, stream=side)
    else:
        f = hab.rotary_frequencies(64, device="cuda")
        o = hab.rotary_append(plan, b.q, None, None, None, None, None, f, stream=side)
    plan.upload()
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not side.query(), "the queue ran empty before the memory was asked for"
    # (only asked for, never written: where it is the plan's, the call has lost it)
    assert all(t.data_ptr() + size <= at or at + size <= t.data_ptr() for t in others)
    torch.cuda.synchronize()
    if call == "attention":
        assert torch.equal(o, want)


def test_nothing_to_keep():
    """A plan of no tokens, never uploaded, on a stream."""
    b = Batch([0, 0], [5, 0])
    assert hab.paged_attention(plan_of(b), b.q, b.k, b.v, b.pages, stream=torch.cuda.Stream()).shape == (0, 512)


def test_an_upload_is_not_captured():
    """A graph would copy out of staging that later uploads have written again:
    refused, with the capture and the plan as they were."""
    b = Batch([1, 40], [300, 90], seed=2)
    want = run(b)
    plan = plan_of(b).upload().upload()
    o = torch.empty_like(b.q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(hab.LoraError, match="captured"):
            plan.upload(ws=plan.ws)
        hab.paged_attention(plan, b.q, b.k, b.v, b.pages, o=o)
    for _ in range(3):
        o.zero_()
        plan.rebuild(b.new, b.kv).upload(ws=plan.ws)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        assert torch.equal(hab.paged_attention(plan, b.q, b.k, b.v, b.pages), want)
