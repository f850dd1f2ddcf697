"""Scores of -inf: a row whose keys all score so has no weights (NaN, as
exp(-inf + inf) is), and is told apart from a row that sees no key (zeros)."""
import math

import pytest
import torch

import heterogeneous_adapter_batching_amd as hab
from attention_reference import Batch
from test_gpu_attention import check, run

pytestmark = pytest.mark.gpu


def batch(new, kv, lost, dtype="bf16", heads=4, kv_heads=2, **kw):
    """A batch whose keys `lost` (a set of places for each sequence) score -inf
    with every query; its 64-bit form leaves them out: a weight of zero."""
    b = Batch(new, kv, heads=heads, kv_heads=kv_heads, dtype=dtype, **kw)
    b.q.view(b.tokens, heads, b.dim)[..., 0] = 1.0
    for s, places in enumerate(lost):
        at = torch.tensor(sorted(places), dtype=torch.int64, device="cuda")
        page = b.pages[s, at // b.page].long()
        ok = (page >= 0) & (page < b.k.shape[0])
        b.k[page[ok], :, (at % b.page)[ok], 0] = -math.inf
    whole = type(b).seen
    kept = [torch.tensor([j not in p for j in range(n)], dtype=torch.bool, device="cuda")
            for p, n in zip(lost, b.kv)]
    b.sees = lambda s: whole(b, s)
    b.seen = lambda s: whole(b, s) & kept[s]
    return b


def check_rows(b, o):
    """Rows that see only lost keys are NaN in every element, the others right
    (those of no key at all: zeros)."""
    for s, part in enumerate(o.split(b.new)):
        rows = b.pages[s, :-(-b.kv[s] // b.page)]
        there = ((rows >= 0) & (rows < b.k.shape[0])).repeat_interleave(b.page)[:b.kv[s]]
        nothing = (b.sees(s) & there).any(1) & ~(b.seen(s) & there).any(1)
        assert part[nothing].isnan().all(), s
        part[nothing] = 0.0                      # (what the 64-bit form has there)
        assert not part.isnan().any(), s
    check(b, o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 4, 40, 200])
def test_all_keys(new, dtype):
    b = batch([new, 1], [new + 30, 9], [range(new + 30), ()], dtype)
    o = run(b)
    assert o[:new].isnan().all() and not o[new:].isnan().any()
    check_rows(b, o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [3, 50, 200])
def test_first_keys_of_a_prompt(new, dtype):
    """The first tokens see the lost keys alone; later ones see others too."""
    for lost in (1, 2, min(new - 1, 70)):
        check_rows(b := batch([new], [new], [range(lost)], dtype, seed=lost), run(b))
        assert not b.seen(0).any(1)[:lost].any() and b.seen(0).any(1)[lost:].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 40])
def test_parts(new, dim, dtype):
    """Contexts in several parts: lost in all of them, in all but one key, in
    some whole parts, and in one part alone."""
    n = 6000
    for lost in (range(n), set(range(n)) - {n // 2}, range(0, 3000), range(3000, n - new),
                 range(1000, 2000)):
        b = batch([new], [n], [lost], dtype, dim=dim, page=64, heads=2, kv_heads=1)
        check_rows(b, run(b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40])
def test_windows(new, dtype):
    """Rows whose window holds lost keys alone."""
    b = batch([new], [300], [range(300 - new - 60, 300 - new // 2)], dtype, window=20)
    assert not b.seen(0).any(1)[0]
    check_rows(b, run(b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new, kv", [(1, 200), (40, 200), (1, 6000), (40, 6000)])
def test_beside_pages_that_are_none(new, kv, dtype):
    """Absent keys and lost ones: NaN where a lost one is seen, zeros where
    every key is absent."""
    lost = batch([new, new], [kv, kv], [range(kv), ()], dtype, page=64)
    lost.pages[0, 1:] = -1
    lost.pages[1, :] = lost.k.shape[0]
    o = run(lost)
    assert o[:new].isnan().all() and (o[new:] == 0).all()


@pytest.mark.parametrize("new", [1, 40])
def test_an_encoder_without_states(new):
    b = batch([new, new], [0, 70], [(), range(70)], causal=False)
    o = run(b)
    assert (o[:new] == 0).all() and o[new:].isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40])
def test_products_that_overflow(new, dtype):
    """Finite queries and keys whose float32 product is -inf, for every key."""
    b = Batch([new], [90], dtype=dtype)
    b.q.fill_(3e38)
    b.k.copy_(torch.where(b.k.isnan(), b.k, torch.full_like(b.k, -3e38)))
    assert run(b).isnan().all()


def test_replayed():
    """A captured decode step whose keys are lost at one replay and not at the
    next."""
    b = batch([1, 1], [700, 50], [(), ()], page=64)
    plan = hab.AttentionPlan(b.heads, b.kv_heads, b.dim, b.page, b.new, b.kv, max_kv=704).upload()
    o, clean = torch.empty_like(b.q), b.k.clone()
    pages = torch.zeros(2, 11, dtype=torch.int32, device="cuda")
    pages[:, :b.pages.shape[1]] = b.pages
    hab.paged_attention(plan, b.q, b.k, b.v, pages, o=o)
    want = o.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hab.paged_attention(plan, b.q, b.k, b.v, pages, o=o)
    for _ in range(3):
        b.k[..., 0] = -math.inf
        graph.replay()
        torch.cuda.synchronize()
        assert o.isnan().all()
        b.k.copy_(clean)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
