"""Rotary positions into a paged cache against their definition in 64 bits."""
import math

import pytest
import torch

import heterogeneous_adapter_batching_amd as hab
from attention_reference import DTYPES, Batch

pytestmark = pytest.mark.gpu


def case(new, kv, dtype="bf16", seed=0, **kw):
    b = Batch(new, kv, dtype=dtype, seed=seed, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rows = torch.randn(b.tokens, (b.heads + 2 * b.kv_heads) * b.dim, generator=g,
                       device="cuda").to(DTYPES[dtype])
    n, m = b.heads * b.dim, b.kv_heads * b.dim
    return b, *rows.split([n, m, m], 1)


def plan_of(b):
    return hab.AttentionPlan(b.heads, b.kv_heads, b.dim, b.page, b.new, b.kv, dtype=b.dtype,
                             causal=b.causal).upload()


def check(b, rows, heads, got, positions, freqs, layout, magnitude):
    """Off by the output's half step, and float32's roundings of the sine and
    cosine (2 half steps of theirs and 2^-23 of the turn's fraction times 2 pi:
    at most 2^-20), the products and the sum, relative to |x| + |y|."""
    want = b.turned(rows, heads, positions, freqs, layout, magnitude)
    r = 0 if freqs is None else 2 * freqs.shape[0]
    x = rows.double().reshape(want.shape)[..., :r].abs()
    if layout == "half":
        size = (x[..., :r // 2] + x[..., r // 2:]).repeat(1, 1, 2)
    else:
        size = (x[..., 0::2] + x[..., 1::2]).repeat_interleave(2, -1)
    tol = torch.finfo(DTYPES[b.dtype]).eps / 2 * want.abs()
    tol[..., :r] += size * abs(magnitude) * 2.0 ** -20
    off = (got.double().reshape(want.shape) - want).abs()
    assert (off <= tol).all(), (off / tol).max()
    assert torch.equal(got.reshape(want.shape)[..., r:], rows.reshape(want.shape)[..., r:])


def run(b, q, k, v, freqs, layout="half", magnitude=1.0, positions=None, **kw):
    """Rotates and appends, and checks every place of the cache."""
    kc, vc = b.k.clone(), b.v.clone()
    out = hab.rotary_append(plan_of(b), q, k, v, kc, vc, b.pages, freqs, layout=layout,
                            magnitude=magnitude, positions=positions, **kw)
    pos, page, slot = b.places()
    at = pos if positions is None else positions[:b.tokens]
    check(b, q, b.heads, out[:b.tokens], at, freqs, layout, magnitude)
    check(b, k, b.kv_heads, kc[page, :, slot], at, freqs, layout, magnitude)
    assert torch.equal(vc[page, :, slot].flatten(1), v)
    for before, after in ((b.k, kc), (b.v, vc)):
        same = (before == after) | (before.isnan() & after.isnan())
        same[page, :, slot] = True
        assert same.all()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim, part", [(128, 128), (128, 64), (64, 64), (80, 80), (80, 32), (72, 72),
                                       (40, 20), (128, 30), (8, 2), (256, 256), (96, 24), (104, 88)])
def test_parts_of_a_head(dim, part, layout, dtype):
    f = hab.rotary_frequencies(part, device="cuda")
    run(*case([1, 5, 30, 0, 2], [40, 5, 100, 3, 19], dtype, dim, dim=dim), f, layout)


@pytest.mark.parametrize("order", ["heads", "tokens", "joined"])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_pages_and_strides(page, order):
    f = hab.rotary_frequencies(64, device="cuda")
    run(*case([1, 70, 20], [17, 170, 20], seed=page, page=page, order=order), f)


@pytest.mark.parametrize("scaling", ["none", "linear", "by_parts"])
def test_far_positions(scaling):
    """Angles keep their fraction of a turn at positions of millions."""
    b, q, k, v = case([3, 4], [30, 4], "f32", 1, dim=128)
    f = hab.rotary_frequencies(128, base=500000.0, scaling=scaling, factor=8.0, original_length=8192,
                               device="cuda")
    pos = torch.tensor([0, 1, 131071, 1 << 20, 10_000_019, (1 << 31) - 1, 77], dtype=torch.int32,
                       device="cuda")
    run(b, q, k, v, f, magnitude=1.2, positions=pos)
    run(b, q, k, v, f, "interleaved", positions=pos)


def test_frequencies():
    """The three kinds against their definitions."""
    f = hab.rotary_frequencies(64, base=10000.0)
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert torch.allclose(f, want, rtol=1e-14, atol=0)
    g = hab.rotary_frequencies(64, base=10000.0, scaling="linear", factor=4.0)
    assert torch.allclose(g, want / 4, rtol=1e-14, atol=0)
    h = hab.rotary_frequencies(64, base=10000.0, scaling="by_parts", factor=4.0, original_length=4096,
                               low=1.0, high=32.0)
    turns = want * 4096 / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    assert torch.allclose(h, want * keep + want / 4 * (1 - keep), rtol=1e-14, atol=0)
    assert h[0] == f[0] and h[-1] == f[-1] / 4


@pytest.mark.parametrize("layout, part", [("half", 64), ("interleaved", 64), ("half", 20),
                                          ("interleaved", 12)])
def test_in_place(layout, part):
    b, q, k, v = case([1, 40], [9, 70], seed=2)
    f = hab.rotary_frequencies(part, device="cuda")
    want = hab.rotary_append(plan_of(b), q, None, None, None, None, None, f, layout=layout)
    assert hab.rotary_append(plan_of(b), q, k, v, b.k, b.v, b.pages, f, layout=layout, q_out=q) is q
    assert torch.equal(q, want)


def test_keys_and_values_alone():
    """An encoder's states into their pages, unrotated, without queries."""
    b, q, k, v = case([33, 5], [33, 5], seed=3, causal=False)
    out = hab.rotary_append(plan_of(b), None, k, v, b.k, b.v, b.pages, None)
    pos, page, slot = b.places()
    assert out is None
    assert torch.equal(b.k[page, :, slot].flatten(1), k)
    assert torch.equal(b.v[page, :, slot].flatten(1), v)


def test_pages_that_are_none():
    """A token whose page is outside the cache is rotated and not stored."""
    b, q, k, v = case([1, 1, 20], [9, 30, 40], seed=4)
    f = hab.rotary_frequencies(64, device="cuda")
    b.pages[0, 0], b.pages[2, 1] = b.k.shape[0], -1
    kc, vc = b.k.clone(), b.v.clone()
    out = hab.rotary_append(plan_of(b), q, k, v, kc, vc, b.pages, f)
    pos, page, slot = b.places()
    check(b, q, b.heads, out, pos, f, "half", 1.0)
    kept = (page >= 0) & (page < b.k.shape[0])
    assert kept.sum() == 1 + 8
    check(b, k[kept], b.kv_heads, kc[page[kept], :, slot[kept]], pos[kept], f, "half", 1.0)
    same = (b.v == vc) | (b.v.isnan() & vc.isnan())
    same[page[kept], :, slot[kept]] = True
    assert same.all()


def test_rows_past_the_batch():
    """A padded batch: rows past the plan's tokens are neither read nor written."""
    b, q, k, v = case([1, 3], [8, 50], seed=5)
    f = hab.rotary_frequencies(64, device="cuda")
    rows = torch.cat([t for t in (q, k, v)], 1)
    padded = torch.cat([rows, torch.full((4, rows.shape[1]), math.nan, dtype=rows.dtype, device="cuda")])
    n, m = q.shape[1], k.shape[1]
    q2, k2, v2 = padded.split([n, m, m], 1)
    out = torch.full((b.tokens + 4, n), 5.0, dtype=q.dtype, device="cuda")
    kc, vc = b.k.clone(), b.v.clone()
    hab.rotary_append(plan_of(b), q2, k2, v2, kc, vc, b.pages, f, q_out=out)
    assert (out[b.tokens:] == 5).all()
    assert torch.equal(out[:b.tokens], run(b, q, k, v, f))


def test_captured_and_replayed():
    b, q, k, v = case([1, 1, 20], [9, 30, 40], seed=6)
    q, k, v = q.clone(), k.clone(), v.clone()
    f = hab.rotary_frequencies(64, device="cuda")
    plan, out = plan_of(b), torch.empty_like(q)
    kc, vc = b.k.clone(), b.v.clone()
    args = (plan, q, k, v, kc, vc, b.pages, f)
    hab.rotary_append(*args, q_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hab.rotary_append(*args, q_out=out)
    for s in range(3):
        for t in (q, k, v):
            t.normal_()
        graph.replay()
        torch.cuda.synchronize()
        pos, page, slot = b.places()
        check(b, q, b.heads, out, pos, f, "half", 1.0)
        check(b, k, b.kv_heads, kc[page, :, slot], pos, f, "half", 1.0)
        assert torch.equal(vc[page, :, slot].flatten(1), v)


def test_replayed_with_fewer_keys_than_new_tokens():
    """A plan that is not causal may be rebuilt so, and a captured append
    replayed: tokens in front of the first key are not stored."""
    b, q, k, v = case([2, 3], [9, 30], seed=7, causal=False)
    plan = hab.AttentionPlan(b.heads, b.kv_heads, b.dim, b.page, b.new, b.kv, dtype=b.dtype,
                             causal=False, max_kv=30).upload()
    k, v = k.clone(), v.clone()
    page = b.page
    kc = torch.zeros(8, b.kv_heads, page, b.dim, dtype=k.dtype, device="cuda")
    vc = torch.zeros_like(kc)
    pages = torch.tensor([[3, 5], [6, 2]], dtype=torch.int32, device="cuda")[:, :max(1, -(-30 // page))]
    hab.rotary_append(plan, None, k, v, kc, vc, pages, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hab.rotary_append(plan, None, k, v, kc, vc, pages, None)
    plan.rebuild([2, 3], [1, 30]).upload(ws=plan.ws)
    for _ in range(3):
        kc.zero_()
        vc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for c, rows in ((kc, k), (vc, v)):
            want = torch.zeros_like(c)
            want[3, :, 0] = rows[1].view(b.kv_heads, b.dim)
            for i, pos in enumerate((27, 28, 29)):
                want[int(pages[1, pos // page]), :, pos % page] = rows[2 + i].view(b.kv_heads, b.dim)
            assert torch.equal(c, want)
