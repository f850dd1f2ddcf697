"""Attention over a paged cache against its definition in 64 bits."""
import math

import pytest
import torch

import heterogeneous_adapter_batching_amd as hab
from attention_reference import DTYPES, Batch

pytestmark = pytest.mark.gpu

# What rounding a weight costs where its remainder enters the product too (few
# rows), and where it does not (prompts); float32 keeps it.
FEW, PROMPT = 2.0 ** -16, 2.0 ** -8


def plan_of(b, **kw):
    return hab.AttentionPlan(b.heads, b.kv_heads, b.dim, b.page, b.new, b.kv, dtype=b.dtype,
                             causal=b.causal, window=b.window, **kw)


def check(b, got, scale=None, eps=None):
    o, mean, size = b.attention(scale)
    if eps is None:
        eps = 0.0 if b.dtype == "f32" else \
            FEW if max(b.new + [0]) * b.heads // b.kv_heads <= 16 else PROMPT
    tol = b.tolerance(o, mean, size, eps)
    off = (got.double().reshape(o.shape) - o).abs()
    assert torch.isfinite(got).all()
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{worst} times the tolerance"


def run(b, **kw):
    return hab.paged_attention(plan_of(b).upload(), b.q, b.k, b.v, b.pages, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 128, 136, 256])
def test_single_tokens(dim, dtype):
    """A decode step over contexts from one key to several parts."""
    check(b := Batch([1] * 7, [1, 2, 15, 16, 17, 300, 2500], dim=dim, dtype=dtype, seed=dim), run(b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads, kv_heads", [(1, 1), (5, 5), (6, 2), (8, 1), (21, 3), (24, 1), (40, 1),
                                             (64, 1)])
def test_head_groups(heads, kv_heads, dtype):
    """Rows of one key head below, at and past a tile of 16."""
    check(b := Batch([1, 1, 2], [33, 700, 64], heads=heads, kv_heads=kv_heads, dtype=dtype,
                     seed=heads), run(b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new, kv", [
    ([3], [3]), ([5, 1, 9], [5, 40, 100]), ([16], [16]), ([17, 33], [17, 95]), ([64], [64]),
    ([65], [200]), ([130, 1, 0, 7], [130, 513, 20, 7]), ([300], [1300]), ([257, 255], [257, 900]),
])
def test_chunks(new, kv, dtype):
    """Chunks behind cached keys and alone, short ones and single tokens among
    them, one sequence without new tokens."""
    check(b := Batch(new, kv, dtype=dtype, seed=len(new) + kv[0]), run(b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [16, 80, 96, 128, 192, 256])
def test_chunks_of_wide_heads(dim, dtype):
    check(b := Batch([70, 40, 1], [70, 333, 90], dim=dim, dtype=dtype, heads=6, kv_heads=3, seed=dim),
          run(b))


@pytest.mark.parametrize("page", [16, 48, 64, 80, 256])
def test_pages(page):
    """Pages that end inside a tile of keys, and longer than a sequence."""
    b = Batch([1, 90, 20], [page + 1, 3 * page + 90, 20], page=page, seed=page)
    check(b, run(b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 7, 64, 100, 5000])
def test_window(window, dtype):
    check(b := Batch([1, 150, 1, 6], [2000, 420, 3, 90], window=window, dtype=dtype, seed=window),
          run(b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_all_keys(dtype):
    """An encoder's states, fewer and more than the queries; none at all gives
    zeros."""
    b = Batch([1, 40, 3, 200, 5], [700, 5, 0, 130, 1], causal=False, dtype=dtype, heads=4,
              kv_heads=4, seed=3)
    o = run(b)
    check(b, o)
    assert (o[41:44] == 0).all()


@pytest.mark.parametrize("order", ["tokens", "joined"])
@pytest.mark.parametrize("new", [[1, 1], [100, 2]])
def test_cache_strides(order, new):
    """Tokens ahead of heads in memory, keys and values in one tensor."""
    b = Batch(new, [170, 90], order=order, seed=8)
    assert not b.k.is_contiguous()
    check(b, run(b))


def test_queries_and_outputs_in_wider_rows():
    """q as a slice of a product's rows, o as columns of a wider tensor; the
    columns beside it and the rows past the batch stay."""
    b = Batch([1, 33, 1], [50, 80, 7], seed=5)
    wide = torch.full((b.tokens + 5, b.q.shape[1] + 48), 7.0, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(b.tokens + 5, b.q.shape[1] + 256, device="cuda").to(torch.bfloat16)
    rows[:b.tokens, 64:64 + b.q.shape[1]] = b.q
    rows[b.tokens:] = math.nan
    o = wide[:, 16:16 + b.q.shape[1]]
    out = hab.paged_attention(plan_of(b).upload(), rows[:, 64:64 + b.q.shape[1]], b.k, b.v, b.pages,
                              o=o)
    assert out is o
    check(b, o[:b.tokens].contiguous())
    assert (wide[b.tokens:] == 7).all() and (wide[:, :16] == 7).all() and (wide[:, -32:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("window", [0, 9])
def test_values_that_a_token_does_not_see(bad, window, dtype):
    """Infinities and NaN in later keys and values of the same chunk, and ahead
    of the window, stay away from the tokens that do not see them."""
    for new, kv in (([4], [40]), ([200], [300])):
        b = Batch(new, kv, window=window, dtype=dtype, seed=11, heads=4, kv_heads=2)
        clean = run(b)
        at = kv[0] - new[0] + 2                  # the third new token's own
        page, slot = int(b.pages[0, at // b.page]), at % b.page
        b.k[page, :, slot, 3], b.v[page, :, slot, 5] = bad, bad
        o = run(b)
        hit = b.seen(0)[:, at]
        assert hit.sum() > 0 and (~hit).sum() > 0
        assert torch.equal(o[~hit], clean[~hit])
        assert not torch.isfinite(o[hit].reshape(-1, b.heads, b.dim)[..., 5]).any()


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 4.0])
def test_scale(scale):
    """Weights from all alike to a single key's, with scores in the hundreds."""
    b = Batch([1, 60], [900, 60], seed=2, std=3.0)
    check(b, run(b, scale=scale), scale)


def test_scores_past_the_exponent():
    """Scores of thousands: the running maximum keeps the sums in range."""
    b = Batch([1, 70], [600, 500], seed=4, std=200.0, dtype="f32")
    check(b, run(b))


@pytest.mark.parametrize("new", [[1, 1], [80, 1]])
def test_pages_that_are_none(new):
    """Numbers outside the cache in the table: their keys count as absent."""
    b = Batch(new, [200, 170], seed=6)
    b.pages[0, 3], b.pages[0, 7], b.pages[1, 0] = -1, b.k.shape[0], 1 << 30
    check(b, run(b))
    b.pages[1, :] = -5
    o = run(b)
    assert (o[-1] == 0).all()


def test_one_sequence_much_longer_than_the_others():
    """The parts of a long context beside short ones (and a long one beside a
    prompt)."""
    check(b := Batch([1] * 9, [40000] + [50] * 8, seed=9, page=64), run(b))
    check(b := Batch([1, 300], [20000, 300], seed=9, page=64, dim=128, heads=8), run(b))


@pytest.mark.parametrize("bad", [None, math.nan])
def test_units_of_more_than_64_tiles(bad):
    """Chunks whose workgroups look their pages up more than once: more work
    than the launch cuts (unless for a value that sends them again)."""
    b = Batch([40, 17, 33, 64], [18000, 17999, 9000, 90], heads=64, kv_heads=64, dim=16, page=48, seed=20)
    clean = run(b)
    check(b, clean)
    if bad is not None:
        at = b.kv[0] - 3                         # seen by the last three tokens alone
        b.v[int(b.pages[0, at // b.page]), :, at % b.page, 7] = bad
        o = run(b)
        keep = torch.ones(b.tokens, dtype=torch.bool, device="cuda")
        keep[37:40] = False
        assert torch.equal(o[keep], clean[keep])
        assert o[37:40].view(3, 64, 16)[..., 7].isnan().all()


@pytest.mark.parametrize("dim", [24, 128, 200])
@pytest.mark.parametrize("seqs", [11, 16])
def test_many_float32_chunks(dim, seqs):
    """Batches that fill the chip with tiles of 32 and 64 rows."""
    check(b := Batch([70] * seqs, [70 + 13 * s for s in range(seqs)], heads=8, kv_heads=8, dim=dim,
                     dtype="f32", seed=dim), run(b))


@pytest.mark.parametrize("new", [[3, 1], [120, 2]])
def test_padded_queries(new):
    """Rows past the plan's tokens: not read, and zeros in a new output."""
    b = Batch(new, [200, 50], seed=21)
    q = torch.full((b.tokens + 6, b.q.shape[1]), math.nan, dtype=torch.bfloat16, device="cuda")
    q[:b.tokens] = b.q
    o = hab.paged_attention(plan_of(b).upload(), q, b.k, b.v, b.pages)
    check(b, o[:b.tokens])
    assert (o[b.tokens:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_query_that_is_not_finite(dtype):
    for new, kv in (([4], [40]), ([200], [300])):
        b = Batch(new, kv, dtype=dtype, seed=22)
        clean = run(b)
        b.q[1, 70], b.q[2, 3] = math.nan, math.inf
        o = run(b).view(b.tokens, b.heads, b.dim)
        assert o[1, 1].isnan().all() and not torch.isfinite(o[2, 0]).any()
        keep = torch.ones(b.tokens, b.heads, dtype=torch.bool, device="cuda")
        keep[1, 1] = keep[2, 0] = False
        assert torch.equal(o[keep], clean.view(o.shape)[keep])


def test_deterministic():
    b = Batch([1, 200, 1], [5000, 700, 90], seed=10)
    a = run(b)
    for _ in range(3):
        assert torch.equal(run(b), a)


def test_a_cache_past_four_gib():
    """Pages whose elements lie past 2^32 bytes."""
    page, dim, pages = 64, 128, (1 << 32) // (64 * 128 * 2) + 40
    k = torch.zeros(pages, 1, page, dim, dtype=torch.bfloat16, device="cuda")
    b = Batch([1, 90], [150, 300], heads=4, kv_heads=1, dim=dim, page=page, seed=12)
    moved = b.pages.clone()
    moved[b.pages >= 0] += pages - b.k.shape[0]
    v = torch.zeros_like(k)
    k[-b.k.shape[0]:], v[-b.k.shape[0]:] = b.k, b.v
    plan = plan_of(b).upload()
    check(b, hab.paged_attention(plan, b.q, k, v, moved))


def test_empty_batches():
    for new, kv in (([], []), ([0, 0], [5, 0])):
        b = Batch(new, kv)
        assert run(b).shape == (0, 512)


def test_rebuilt_plan():
    """The next step's batch in the same plan and workspace."""
    b = Batch([1] * 3, [40, 700, 9], seed=13)
    plan = plan_of(b)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    check(b, hab.paged_attention(plan.upload(ws=ws), b.q, b.k, b.v, b.pages))
    for new, kv in (([1] * 3, [41, 701, 10]), ([5, 1], [77, 2100]), ([90], [90])):
        b = Batch(new, kv, seed=14)
        plan.rebuild(b.new, b.kv).upload(ws=ws)
        check(b, hab.paged_attention(plan, b.q, b.k, b.v, b.pages))


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 1, 3]])
def test_captured_and_replayed_with_other_lengths(new):
    """A graph captured with max_kv keeps its launches: replayed after the plan
    was rebuilt for longer sequences, with eager work in between."""
    first = Batch(new, [n + 20 for n in new], seed=15, page=64)
    plan = plan_of(first, max_kv=6000).upload()
    q, o = first.q.clone(), torch.empty_like(first.q)
    k = torch.zeros(400, first.kv_heads, 64, first.dim, dtype=torch.bfloat16, device="cuda")
    v, pages = torch.zeros_like(k), torch.zeros(len(new), 94, dtype=torch.int32, device="cuda")

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
    for kv in ([5000, 60, 777], [45, 6000, 3], [3000, 2999, 64], [6000, 6000, 6000]):
        b = Batch(new, kv, seed=kv[0], page=64)
        fill(b)
        plan.rebuild(b.new, b.kv).upload(ws=plan.ws)
        o.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        check(b, o)
        eager = hab.paged_attention(plan, q, k, v, pages)
        assert torch.equal(eager, o)


def test_two_streams():
    """Two plans at once on streams of their own, tensors made on another."""
    batches = [Batch([1, 120, 1], [3000, 400, 77], seed=s) for s in (16, 17)]
    want = [run(b) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    plans = [plan_of(b).upload() for b in batches]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for b, s, p, g in zip(batches, streams, plans, got):
            g.append(hab.paged_attention(p, b.q, b.k, b.v, b.pages, stream=s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


def test_the_same_page_twice():
    """Two sequences that share their first pages."""
    b = Batch([1, 30], [100, 160], seed=18)
    b.pages[1, :6] = b.pages[0, :6]
    check(b, run(b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_random_batches(dtype):
    import random
    r = random.Random(19)
    for i in range(24):
        kv_heads, group = r.choice([1, 2, 3]), r.choice([1, 2, 4, 5, 12])
        new = [r.choice([0, 1, 1, 2, r.randrange(1, 180)]) for _ in range(r.randrange(1, 7))]
        kv = [n + r.choice([0, 1, r.randrange(0, 900)]) for n in new]
        causal = r.random() < 0.75
        b = Batch(new, kv, heads=kv_heads * group, kv_heads=kv_heads, dim=8 * r.randrange(1, 33),
                  page=16 * r.randrange(1, 9), dtype=dtype, causal=causal,
                  window=r.randrange(1, 300) if causal and r.random() < 0.4 else 0, seed=i)
        print(i, new, kv, b.heads, b.kv_heads, b.dim, b.page, causal, b.window, flush=True)
        check(b, run(b))
