"""float32 batches that fill the chip with tiles of 32 and 64 rows: what the
masks leave of a tile's 16-row parts, and keys read more than once (smaller
batches take tiles of 16 rows, whatever their lengths)."""
import math

import pytest
import torch

import heterogeneous_adapter_batching_amd as hab
from attention_reference import Batch
from test_gpu_attention import check, plan_of, run
from test_gpu_attention_infinite_scores import batch, check_rows

pytestmark = pytest.mark.gpu

SEQS = {64: 16, 32: 11}          # of 70 tokens, 8 heads: 256 tiles of 64 rows; 264 of 32 (176 of 64)


def tile_rows(b, plan=None):
    """The rows of a tile that the batch's plan took (its units, where no tile is
    in several parts)."""
    stats = (plan or plan_of(b)).stats()
    assert stats["joins"] == 0
    group = b.heads // b.kv_heads
    return [r for r in (16, 32, 64)
            if sum(-(-n * group // r) for n in b.new) * b.kv_heads == stats["units"]][0]


def make(rows, lens=None, kind=Batch, **kw):
    seqs = SEQS[rows]
    kw = dict(dict(heads=8, kv_heads=8, dim=64, dtype="f32"), **kw)
    b = kind([70] * seqs, [(lens or (lambda s: 70 + 11 * s))(s) for s in range(seqs)], **kw)
    assert tile_rows(b) == rows
    return b


SHAPES = [(64, 64), (64, 128), (32, 40), (32, 128), (32, 200)]


@pytest.mark.parametrize("rows, dim", SHAPES)
@pytest.mark.parametrize("window", [1, 9, 100])
def test_window(rows, dim, window):
    check(b := make(rows, dim=dim, window=window, seed=window), run(b))


@pytest.mark.parametrize("rows, dim", SHAPES)
def test_all_keys(rows, dim):
    b = make(rows, lambda s: (0, 1, 15, 64, 200)[s % 5], dim=dim, causal=False, seed=1)
    o = run(b)
    check(b, o)
    assert (o[:70] == 0).all()


@pytest.mark.parametrize("rows, dim", SHAPES)
@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_a_token_does_not_see(rows, dim, window, bad):
    """Infinities and NaN in keys and values that some rows of a tile see, in
    each of its 16-row parts and behind the first tile."""
    b = make(rows, dim=dim, window=window, seed=2)
    clean = run(b)
    hit = torch.zeros(b.tokens, dtype=torch.bool, device="cuda")
    for s, token in enumerate([3, 20, 40, 60, 66, 69]):
        at = b.kv[s] - 70 + token
        page, slot = int(b.pages[s, at // b.page]), at % b.page
        b.k[page, :, slot, 3], b.v[page, :, slot, 5] = bad, bad
        hit[70 * s:70 * (s + 1)] = b.seen(s)[:, at]
    o = run(b)
    assert torch.equal(o[~hit], clean[~hit])
    assert not torch.isfinite(o[hit].reshape(-1, b.heads, b.dim)[..., 5]).any()


@pytest.mark.parametrize("rows, dim", SHAPES)
def test_pages_that_are_none(rows, dim):
    b = make(rows, dim=dim, seed=3)
    b.pages[0, 0], b.pages[1, 3], b.pages[2, 1] = -1, b.k.shape[0], 1 << 30
    b.pages[3, :] = -5
    o = run(b)
    check(b, o)
    assert (o[210:280] == 0).all()


@pytest.mark.parametrize("rows, dim", SHAPES)
def test_scores_of_minus_infinity(rows, dim):
    seqs = SEQS[rows]
    lost = [range(3 * s) for s in range(seqs)]
    lost[1], lost[2] = range(81), range(20, 50)
    b = batch([70] * seqs, [70 + 11 * s for s in range(seqs)], lost, "f32", heads=8, kv_heads=8, dim=dim)
    assert tile_rows(b) == rows
    check_rows(b, run(b))


@pytest.mark.parametrize("window", [0, 33])
def test_head_groups(window):
    """Rows of a token on both sides of a tile's end."""
    for seqs, rows, heads, kv_heads in ((32, 64, 6, 2), (19, 32, 6, 2), (20, 64, 15, 3)):
        b = Batch([70] * seqs, [70 + 5 * s for s in range(seqs)], heads=heads, kv_heads=kv_heads,
                  dtype="f32", dim=72, window=window, seed=seqs)
        assert tile_rows(b) == rows
        check(b, run(b))


@pytest.mark.parametrize("rows, dim", SHAPES)
def test_parts(rows, dim):
    """Tiles of many rows whose keys are in several parts."""
    b = Batch([70] * SEQS[rows], [70 + 300 * s for s in range(SEQS[rows])], heads=8, kv_heads=8, dim=dim,
              page=64, dtype="f32", seed=4)
    assert plan_of(b).stats()["joins"] > 100
    check(b, run(b))


@pytest.mark.parametrize("rows, dim", SHAPES)
def test_captured_and_replayed_with_other_lengths(rows, dim):
    seqs = SEQS[rows]
    first = make(rows, dim=dim, seed=5, page=64)
    plan = plan_of(first, max_kv=1500).upload()
    q, o = first.q.clone(), torch.empty_like(first.q)
    k = torch.zeros(seqs * 24 + 2, 8, 64, dim, device="cuda")
    v, pages = torch.zeros_like(k), torch.zeros(seqs, 24, dtype=torch.int32, device="cuda")

    def fill(b):
        q.copy_(b.q)
        k[:b.k.shape[0]], v[:b.v.shape[0]] = b.k, b.v
        pages[:, :b.pages.shape[1]] = b.pages

    fill(first)
    hab.paged_attention(plan, q, k, v, pages, o=o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hab.paged_attention(plan, q, k, v, pages, o=o)
    for most in (1500, 90, 700):
        b = Batch(first.new, [70 + (most - 70) * s // (seqs - 1) for s in range(seqs)], heads=8, kv_heads=8,
                  dim=dim, page=64, dtype="f32", seed=most)
        fill(b)
        plan.rebuild(b.new, b.kv).upload(ws=plan.ws)
        o.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        check(b, o)
        assert torch.equal(hab.paged_attention(plan, q, k, v, pages), o)
