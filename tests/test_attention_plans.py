"""How a plan cuts a few tokens over short contexts (host side, no GPU)."""
import pytest

import heterogeneous_adapter_batching_amd as hab


def stats(tokens, keys, kv_heads=8, dim=128, dtype="bf16", **kw):
    return hab.AttentionPlan(4 * kv_heads, kv_heads, dim, 64, [1] * tokens, [keys] * tokens, dtype=dtype,
                             **kw).stats()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens, kv_heads, whole, parts", [
    (1, 8, 512, 513), (1, 1, 512, 513), (20, 8, 512, 513), (21, 8, 1024, 1025), (32, 8, 1024, 1025),
    (160, 1, 512, 513), (161, 1, 1024, 1025)])
def test_parts_of_short_contexts(tokens, kv_heads, whole, parts, dim, dtype):
    """Whole tiles up to 512 keys, or up to 1024 with more than 160 of them."""
    s = stats(tokens, whole, kv_heads, dim, dtype)
    assert (s["units"], s["joins"]) == (tokens * kv_heads, 0)
    s = stats(tokens, parts, kv_heads, dim, dtype)
    assert s["joins"] == tokens * kv_heads and s["units"] > s["joins"]


def test_other_plans():
    # more tiles than workgroups of 8 waves; heads of 256; room for longer contexts
    assert stats(33, 256)["joins"] == 0 and stats(33, 300)["joins"] == 264
    assert stats(1, 500, dim=256)["joins"] == 8
    assert stats(1, 400, max_kv=512)["joins"] == 0 and stats(1, 400, max_kv=8192)["joins"] == 8
