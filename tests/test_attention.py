"""The attention around the products, host side: plans, and refusals (nothing
is enqueued, so no GPU is needed)."""
import ctypes
import math

import pytest

import heterogeneous_adapter_batching_amd as hab
from heterogeneous_adapter_batching_amd._lib import AttnDesc, KvCache, RotaryDesc

BF16, F32 = 1, 0
EINVAL, EDTYPE, ESTATE = -1, -5, -9
P = 1 << 32   # addresses that no call may reach
M = 1 << 26


def ints(values):
    return (ctypes.c_int32 * max(len(values), 1))(*values)


def create(new=(1, 4), kv=(9, 40), dtype=BF16, heads=8, kv_heads=2, dim=64, page=16, causal=1,
           window=0, max_kv=0, seqs=None, desc=True):
    h = ctypes.c_void_p()
    d = AttnDesc(dtype, heads, kv_heads, dim, page, causal, window, max_kv)
    st = hab.load().attn_plan_create(ctypes.byref(h), ctypes.byref(d) if desc else None, ints(new),
                                     ints(kv), len(new) if seqs is None else seqs)
    return st, h


@pytest.mark.parametrize("bad, status", [
    (dict(desc=False), EINVAL), (dict(dtype=2), EDTYPE), (dict(heads=0), EINVAL),
    (dict(kv_heads=0), EINVAL), (dict(kv_heads=3), EINVAL), (dict(heads=1), EINVAL),
    (dict(heads=2048, kv_heads=2048), EINVAL), (dict(dim=0), EINVAL), (dict(dim=60), EINVAL),
    (dict(dim=264), EINVAL), (dict(page=0), EINVAL), (dict(page=24), EINVAL), (dict(page=8), EINVAL),
    (dict(page=1 << 17), EINVAL), (dict(causal=2), EINVAL), (dict(window=-1), EINVAL),
    (dict(window=5, causal=0), EINVAL), (dict(max_kv=-1), EINVAL), (dict(max_kv=39), EINVAL),
    (dict(seqs=-1), EINVAL), (dict(new=[-1, 1]), EINVAL), (dict(kv=[-1, 40]), EINVAL),
    (dict(kv=[9, 3]), EINVAL), (dict(new=[1 << 23, 1 << 23], kv=[1 << 23, 1 << 23]), EINVAL),
    (dict(new=[1 << 22], kv=[1 << 22], heads=1024, kv_heads=1024), EINVAL),
    (dict(kv=[9, (1 << 30) + 1]), EINVAL), (dict(new=[1 << 24], kv=[1 << 24]), EINVAL),
])
def test_plan_refusals(bad, status):
    st, h = create(**bad)
    assert st == status and not h.value
    assert hab.load().lora_last_error()


def test_plan_of_nothing():
    for new, kv in (((), ()), ((0, 0), (0, 70))):
        st, h = create(new, kv)
        assert st == 0 and hab.load().attn_plan_workspace_bytes(h) >= 256
        hab.load().attn_plan_destroy(h)
    assert hab.load().attn_plan_destroy(None) == 0
    assert hab.load().attn_plan_create(None, None, None, None, 0) == EINVAL
    assert hab.load().attn_plan_workspace_bytes(None) == 0


def test_python_refusals():
    make = lambda *a, **k: hab.AttentionPlan(8, 2, 64, 16, *a, **k)  # noqa: E731
    for new, kv in (([1], [1, 2]), ([1.5], [2]), ([[1]], [[1]]), ([1 << 40], [1 << 40])):
        with pytest.raises(ValueError):
            make(new, kv)
    with pytest.raises(hab.LoraError):
        make([5], [4])
    with pytest.raises(KeyError):
        make([1], [1], dtype="f16")
    with pytest.raises(ValueError):
        hab.AttentionPlan(1 << 33, 2, 64, 16, [1], [1])
    plan = make([5], [4], causal=False)
    with pytest.raises(ValueError):
        plan.rebuild([1, 2], [1])
    for k in (dict(scaling="cubic"), ):
        with pytest.raises(ValueError):
            hab.rotary_frequencies(64, **k)
    for n, k in ((63, {}), (0, {}), (512, {}), (64, dict(base=0.0)), (64, dict(base=math.inf)),
                 (64, dict(scaling="linear", factor=0.0)),
                 (64, dict(scaling="by_parts", factor=2.0)),
                 (64, dict(scaling="by_parts", factor=2.0, original_length=100, low=5, high=5))):
        with pytest.raises(hab.LoraError):
            hab.rotary_frequencies(n, **k)


def units(plan):
    return plan.stats()["units"]


def test_parts():
    """Every tile of rows is a part at least; one long sequence is cut, a batch
    of many is not cut finer than the launch needs; rebuilding re-plans."""
    make = lambda *a, **k: hab.AttentionPlan(32, 8, 128, 64, *a, **k)  # noqa: E731
    assert units(make([1], [1])) == 8 and make([1], [1]).stats()["joins"] == 0
    long = make([1], [100000])
    assert long.stats()["joins"] == 8 and 256 <= units(long) <= 8 + 1024
    many = make([1] * 512, [300] * 512)
    assert units(many) == 8 * 512 and many.stats()["joins"] == 0
    mixed = make([1] * 64, [100000] + [64] * 63)
    assert mixed.stats()["joins"] == 8 and units(mixed) <= 8 * 64 + 1024
    assert units(many.rebuild([1], [1])) == 8 and many.stats()["tokens"] == 1
    assert many.stats()["max_kv"] == 1


@pytest.mark.parametrize("new", [[1] * 5, [1, 40, 0, 3], [300]])
@pytest.mark.parametrize("most", [64, 100, 256, 6000, 100000])
def test_room_for_any_lengths(new, most):
    """With max_kv a plan's workspace, and so what is launched, is the same for
    all lengths."""
    import random
    r = random.Random(most)
    low = [min(n, most) for n in new]
    plan = hab.AttentionPlan(12, 4, 72, 48, low, low, max_kv=most)
    size = plan.workspace_bytes()
    for i in range(50):
        kv = [most if i == 0 else r.choice([n, most, r.randrange(n, most + 1)]) for n in low]
        plan.rebuild(low, kv)
        assert plan.workspace_bytes() == size
    with pytest.raises(hab.LoraError):
        plan.rebuild(low, [most + 1] * len(low))


def cache(k=P + 2 * M, v=P + 3 * M, page=2 * 16 * 64, head=16 * 64, tok=64, pages=100, vtok=64):
    return KvCache(k, v, page, head, tok, page, head, vtok, pages)


def attend(plan=True, q=P, ldq=512, o=P + M, ldo=512, c=None, kv=True, pages=P + 4 * M, ld_pages=3,
           per=3, scale=0.125, **kw):
    st, h = create(**kw)
    assert st == 0
    c = c or cache()
    st = hab.load().paged_attention(h if plan else None, q, ldq, ctypes.byref(c) if kv else None,
                                    pages, ld_pages, per, scale, o, ldo, None)
    hab.load().attn_plan_destroy(h)
    return st


BAD_CACHES = [
    dict(k=0), dict(v=0), dict(k=P + 2 * M + 8), dict(v=P + 3 * M + 2), dict(page=2 * 16 * 64 + 4),
    dict(head=-8), dict(tok=56), dict(vtok=0), dict(tok=66), dict(tok=1 << 27), dict(pages=0),
    dict(pages=-1), dict(page=1 << 41)]


@pytest.mark.parametrize("bad, status", [
    (dict(plan=False), EINVAL), (dict(q=0), EINVAL), (dict(q=P + 8), EINVAL), (dict(ldq=504), EINVAL),
    (dict(ldq=516), EINVAL), (dict(ldq=1 << 41), EINVAL), (dict(o=0), EINVAL), (dict(o=P + M + 2), EINVAL),
    (dict(ldo=510), EINVAL), (dict(o=P), EINVAL), (dict(o=P + 512), EINVAL), (dict(kv=False), EINVAL),
    (dict(o=P + 2 * M + 64), EINVAL), (dict(o=P + 3 * M), EINVAL),
    (dict(pages=0), EINVAL), (dict(pages=P + 4 * M + 2), EINVAL), (dict(ld_pages=2), EINVAL),
    (dict(per=2, ld_pages=2), EINVAL), (dict(per=-1), EINVAL), (dict(scale=math.nan), EINVAL),
    (dict(scale=math.inf), EINVAL), ({}, ESTATE),
] + [(dict(c=cache(**b)), EINVAL) for b in BAD_CACHES])
def test_paged_attention_refusals(bad, status):
    assert attend(**bad) == status
    assert hab.load().lora_last_error()


def test_empty_batches_look_at_nothing():
    st, h = create((0,), (5,))
    lib = hab.load()
    assert lib.paged_attention(h, 0, 0, None, None, 0, 0, 1.0, 0, 0, None) == 0
    d = RotaryDesc(64, 0, 1.0)
    assert lib.rotary_append(h, ctypes.byref(d), P, 0, P, 0, None, 0, None, 0, None, None, 0, 0, None,
                             P, None) == 0
    lib.attn_plan_destroy(h)


def rotary(plan=True, dim=64, layout=0, magnitude=1.0, desc=True, q=P, ldq=768, qo=P + M, ldqo=512,
           k=P + 1024, ldk=768, v=P + 1280, ldv=768, c=None, kv=True, pages=P + 4 * M, ld_pages=3,
           per=3, positions=None, freqs=P + 5 * M, **kw):
    st, h = create(**kw)
    assert st == 0
    c, d = c or cache(), RotaryDesc(dim, layout, magnitude)
    st = hab.load().rotary_append(h if plan else None, ctypes.byref(d) if desc else None, q, ldq, qo,
                                  ldqo, k, ldk, v, ldv, ctypes.byref(c) if kv else None, pages,
                                  ld_pages, per, positions, freqs, None)
    hab.load().attn_plan_destroy(h)
    return st


@pytest.mark.parametrize("bad, status", [
    (dict(plan=False), EINVAL), (dict(desc=False), EINVAL), (dict(dim=0), EINVAL), (dict(dim=63), EINVAL),
    (dict(dim=66), EINVAL), (dict(dim=-2), EINVAL), (dict(layout=2), EINVAL), (dict(layout=-1), EINVAL),
    (dict(magnitude=math.nan), EINVAL), (dict(freqs=None), EINVAL),
    (dict(freqs=None, dim=0, positions=P), EINVAL), (dict(freqs=P + 4), EINVAL),
    (dict(positions=P + 6 * M + 1), EINVAL), (dict(q=0), EINVAL), (dict(q=0, qo=0, kv=False), EINVAL),
    (dict(q=P + 4), EINVAL), (dict(ldq=508), EINVAL), (dict(qo=0), EINVAL), (dict(ldqo=500), EINVAL),
    (dict(qo=P + 16), EINVAL), (dict(qo=P + 2 * M), EINVAL), (dict(kv=False), EINVAL),
    (dict(k=0), EINVAL), (dict(v=0), EINVAL), (dict(ldk=120), EINVAL), (dict(v=P + 1282), EINVAL),
    (dict(k=P + 2 * M + 64), EINVAL), (dict(v=P + 3 * M), EINVAL), (dict(pages=0), EINVAL),
    (dict(ld_pages=1), EINVAL), (dict(per=2, ld_pages=2), EINVAL),
    (dict(causal=0, new=(1, 4), kv=None), EINVAL), ({}, ESTATE), (dict(qo=P, ldqo=768), ESTATE),
    (dict(freqs=None, dim=0), ESTATE), (dict(q=0, qo=0), ESTATE), (dict(kv=False, k=0, v=0), ESTATE),
] + [(dict(c=cache(**b)), EINVAL) for b in BAD_CACHES])
def test_rotary_append_refusals(bad, status):
    if bad.get("kv", True) is None:              # more new tokens than keys
        st, h = create((1, 4), (1, 3), causal=0)
        assert st == 0
        d, c = RotaryDesc(64, 0, 1.0), cache()
        got = hab.load().rotary_append(h, ctypes.byref(d), P, 768, P + M, 512, P + 1024, 768, P + 1280,
                                       768, ctypes.byref(c), P + 4 * M, 3, 3, None, P + 5 * M, None)
        hab.load().attn_plan_destroy(h)
    else:
        got = rotary(**bad)
    assert got == status
    assert hab.load().lora_last_error()


def test_workspace_refusals():
    lib = hab.load()
    st, h = create()
    n = lib.attn_plan_workspace_bytes(h)
    assert n % 256 == 0 and n > 0
    assert lib.attn_plan_upload(None, P, n, None) == EINVAL
    assert lib.attn_plan_upload(h, None, n, None) == EINVAL
    assert lib.attn_plan_upload(h, P + 16, n, None) == EINVAL
    assert lib.attn_plan_upload(h, P, n - 256, None) == ESTATE
    assert lib.attn_plan_rebuild(None, ints([1]), ints([1]), 1) == EINVAL
    assert lib.attn_plan_rebuild(h, None, ints([1]), 1) == EINVAL
    assert lib.attn_plan_rebuild(h, ints([2]), ints([1]), 1) == EINVAL
    assert lib.attn_plan_stats(None, None, None, None, None) == EINVAL
    assert lib.attn_plan_stats(h, None, None, None, None) == 0
    lib.attn_plan_destroy(h)


def test_tensors_on_the_host_are_refused():
    torch = pytest.importorskip("torch")
    plan = hab.AttentionPlan(8, 2, 64, 16, [1], [9])
    q, kc = torch.zeros(1, 512, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    pages = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(TypeError):
        hab.paged_attention(plan, q, kc, kc, pages)
    with pytest.raises(TypeError):
        hab.rotary_append(plan, q, q[:, :128], q[:, :128], kc, kc, pages, None)


@pytest.mark.parametrize("call", [attend, rotary])
@pytest.mark.parametrize("most, status", [(0, ESTATE), (48, ESTATE), (49, EINVAL)])
def test_page_tables_hold_max_kv(call, most, status):
    """A graph is replayed with the table that it was captured with, for up to
    max_kv keys."""
    assert call(max_kv=most) == status


@pytest.mark.parametrize("call", [attend, rotary])
@pytest.mark.parametrize("bad", [
    dict(ldq=1 << 37), dict(ld_pages=1 << 37), dict(c=cache(page=1 << 36, pages=(1 << 31) - 1)),
    dict(c=cache(head=1 << 37))])
def test_extents_stay_within_64_bits(call, bad):
    assert call(**bad) == EINVAL


@pytest.mark.parametrize("places", [dict(page=0), dict(page=56), dict(head=0), dict(head=32),
                                    dict(v=P + 2 * M)])
def test_places_that_coincide_are_read_and_not_written(places):
    assert attend(c=cache(**places)) == ESTATE
    assert rotary(c=cache(**places)) == EINVAL


def test_places_of_one_page_and_one_head():
    """A dimension of one has any stride."""
    assert rotary(c=cache(page=0, pages=1)) == ESTATE
    assert rotary(c=cache(head=0), heads=4, kv_heads=1) == ESTATE


def test_queries_in_the_cache():
    assert rotary(q=P + 2 * M + 64) == EINVAL and rotary(q=P + 3 * M) == EINVAL
