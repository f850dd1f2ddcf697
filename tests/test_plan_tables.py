"""Which plans carry the product's tables (positions, groups), host side."""
import numpy as np
import pytest

import heterogeneous_adapter_batching_amd as hab

T, ADAPTERS = 1000, 7                              # (short groups: no prompt kernel)
MERGE_BLOCK = 224                                  # bytes, of up to 4 tokens


def up(v):
    return (v + 255) // 256 * 256


@pytest.fixture
def pool():
    p = hab.Pool(1, [64], [64], r_max=16, slab_ptr=1 << 30, slab_bytes=1 << 30)
    for i in range(ADAPTERS):
        p.reserve(i, 16, 1.0)
    return p


def segments():
    starts = np.arange(0, T + 1, 4, dtype=np.int32)
    return starts, (np.arange(len(starts) - 1) % ADAPTERS).astype(np.int32)


TABLES = up(16 * (ADAPTERS + 1)) + up(32 * T)      # a group's row is 16 bytes, a position's 32


def test_plans_with_cores_have_none(pool):
    starts, ids = segments()
    plain = hab.Plan(pool, T, starts, ids)
    cores = hab.Plan(pool, T, starts, ids, seg_sigma=ids)
    assert plain.workspace_bytes(1) - cores.workspace_bytes(1) == TABLES
    # cores on rows without an adapter are none
    none = hab.Plan(pool, T, [0, T, T], [-1, 0], seg_sigma=[3, 4])
    assert none.workspace_bytes(1) == hab.Plan(pool, T, [0, T], [-1]).workspace_bytes(1)


def test_merge_plans_have_none(pool):
    starts, ids = segments()
    weighted = hab.Plan(pool, T, starts, ids, seg_weight=np.ones(len(ids), np.float32))
    merge = hab.Plan.merge(pool, T, starts, ids[:, None], np.ones((len(ids), 1), np.float32))
    blocks = up(len(ids) * MERGE_BLOCK)
    assert weighted.workspace_bytes(1) - merge.workspace_bytes(1) == TABLES - blocks


def test_a_rebuilt_plan_has_what_its_batch_needs(pool):
    starts, ids = segments()
    plan = hab.Plan(pool, T, starts, ids)
    first = plan.workspace_bytes(1)
    assert plan.rebuild(T, starts, ids, seg_sigma=ids).workspace_bytes(1) == first - TABLES
    assert plan.rebuild(T, starts, ids).workspace_bytes(1) == first


def test_bound_covers_every_kind(pool):
    starts, ids = segments()
    bound = pool.workspace_bytes(T, len(ids), 1)
    for plan in (hab.Plan(pool, T, starts, ids), hab.Plan(pool, T, starts, ids, seg_sigma=ids)):
        assert plan.workspace_bytes(1) <= bound
