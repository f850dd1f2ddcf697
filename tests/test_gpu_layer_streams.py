"""On the GPU: outputs and workspaces of calls with stream= come from that
stream's memory, and calls on several streams beside eager work on the
current one give the bits of calls alone."""
import pytest

from test_gpu_linear import BF16, Adapted, _gpu, segments  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def owner(t):
    """The stream whose memory holds t."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


def calls(m, x, w, stream):
    import heterogeneous_adapter_batching_amd as hab
    z = hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], x, w, act="silu", stream=stream)
    y = hab.frozen_linear(x, w, act="silu", stream=stream)
    h, u = hab.block_norm(z, y, post="rms", pre="layer", stream=stream)
    return [z, y, h, u]


def test_outputs_belong_to_the_launch_stream():
    T = 96
    starts, ids = segments(3, T, 4, 3)
    m = Adapted(3, T, 520, [264], [8, 16, 64, 32], ids, starts)
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(T, 520, generator=g).to(BF16).cuda(), torch.randn(264, 520, generator=g).to(BF16).cuda()
    want = calls(m, x, w, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = calls(m, x, w, side)
    assert [owner(t) for t in got] == [side.cuda_stream] * 4
    assert all(owner(t) == torch.cuda.current_stream().cuda_stream for t in want)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_beside_work_on_the_current_stream():
    """The current stream keeps making and dropping tensors of the outputs'
    sizes, with reads and writes of them queued."""
    T = 96
    runs = []
    for seed in (31, 32):
        starts, ids = segments(seed, T, 4, 3)
        m = Adapted(seed, T, 520, [264], [8, 16, 64, 32], ids, starts)
        g = torch.Generator().manual_seed(seed)
        x, w = torch.randn(T, 520, generator=g).to(BF16).cuda(), torch.randn(264, 520, generator=g).to(BF16).cuda()
        runs.append((m, x, w, calls(m, x, w, None), torch.cuda.Stream(), []))
    big = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    sums, expect = [], []
    for i in range(20):
        big = big @ big
        big = big / big.abs().max()
        t = torch.full((T, 264), float(i % 7), dtype=BF16, device="cuda")
        big[0, 0] += 0.0 * t[0, 0]
        sums.append(t.float().sum())
        expect.append(float(i % 7) * T * 264)
        del t
        for m, x, w, _, s, got in runs:
            got.append(calls(m, x, w, s))
    torch.cuda.synchronize()
    assert [float(v) for v in sums] == expect
    for _, _, _, want, _, got in runs:
        assert all(torch.equal(a, b) for ts in got for a, b in zip(ts, want))


def test_captured_on_a_forked_stream():
    """A capture whose calls make their outputs and workspaces, on the capturing
    stream and on one forked from it; replayed on new inputs between eager
    calls."""
    T = 100
    starts, ids = segments(5, T, 4, 3)
    m = Adapted(5, T, 1032, [520], [8, 16, 64, 32], ids, starts)
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn(T, 1032, generator=g).to(BF16).cuda(), torch.randn(520, 1032, generator=g).to(BF16).cuda()
    calls(m, x, w, None)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        here = calls(m, x, w, main)
        side.wait_stream(main)
        forked = calls(m, x, w, side)
        main.wait_stream(side)
    for _ in range(3):
        x.copy_(torch.randn(T, 1032, generator=g).to(BF16))
        want = calls(m, x, w, None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got in (here, forked):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
