"""Workspace sizes of the products, host side: no more than a batch can need,
what a given plan needs, and what serves every batch up to a size."""
import numpy as np
import pytest

import heterogeneous_adapter_batching_amd as hab

MIB = 1 << 20


def pool(k, widths, slots=1024, r_max=64, dtype="bf16", adapters=()):
    p = hab.Pool(1, [k] * len(widths), widths, r_max=r_max, dtype=dtype, max_slots=slots,
                 slab_ptr=1 << 30, slab_bytes=1 << 40)
    for i, r in enumerate(adapters):
        p.reserve(i, r, 1.0)
    return p


def plan_of(p, T, seg, n_adapters):
    starts = np.minimum(np.arange(0, T + seg, seg), T).astype(np.int32)
    ids = (np.arange(len(starts) - 1) % n_adapters).astype(np.int32)
    return hab.Plan(p, T, starts, ids)


def operand_bytes(p, T, nproj):
    """v in float32 and the operand's pieces: what every call keeps."""
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    return up(4 * T * nproj * p.r_max) + up((6 if p.dtype == "bf16" else 4) * T * nproj * p.r_max)


def test_a_prompt_needs_no_partial_sums():
    """A gated prompt whose plan runs in one launch keeps the operand alone:
    the size for its plan says so, and the size for any batch is at most one
    part's sums (it runs in parts when thousands of adapters meet)."""
    p = pool(4096, [14336, 14336], adapters=[16] * 8)
    for T in (4096, 16384):
        pl = plan_of(p, T, 512, 8)
        assert hab.sgmv_linear_workspace_bytes(p, T, 14336, 4096, 2, True, plan=pl) == operand_bytes(p, T, 2)
        few = pool(4096, [14336, 14336], slots=8)
        assert hab.sgmv_linear_workspace_bytes(few, T, 14336, 4096, 2, True) == operand_bytes(p, T, 2)
        most = hab.sgmv_linear_workspace_bytes(p, T, 14336, 4096, 2, True) - operand_bytes(p, T, 2)
        assert most <= 4 * T * (28672 + 64) + 256


SHAPES = [(4096, 4096, False), (4096, 14336, True), (14336, 4096, False), (264, 77, False)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k, n, glu", SHAPES)
def test_any_plan_fits_the_size_for_its_tokens(k, n, glu, dtype):
    wide = n * (1 + glu)
    p = pool(k, [max(8, wide // 8 * 8)], slots=300, dtype=dtype, adapters=[(8, 16, 40, 64)[i % 4] for i in range(300)])
    for T in (1, 12, 13, 40, 100, 128, 300, 700, 2048):
        bound = hab.sgmv_linear_workspace_bytes(p, T, n, k, 1, glu)
        for seg, ads in ((1, 300), (1, 1), (3, 50), (64, 8), (512, 2)):
            need = hab.sgmv_linear_workspace_bytes(p, T, n, k, 1, glu, plan=plan_of(p, T, seg, ads))
            assert operand_bytes(p, T, 1) <= need <= bound, (T, seg, ads)
        none = hab.Plan(p, T, [0, T], [-1])
        need = hab.sgmv_linear_workspace_bytes(p, T, n, k, 1, glu, plan=none)
        assert need == operand_bytes(p, T, 1) + hab.linear_workspace_bytes(T, n, k, dtype, glu) <= bound


@pytest.mark.parametrize("k, n, glu", SHAPES)
def test_one_size_for_every_batch_up_to_a_size(k, n, glu):
    """The need is not monotone in the tokens; the size with up_to is the
    largest of them."""
    p = pool(k, [max(8, n // 8 * 8)])
    top = 700
    most = hab.linear_workspace_bytes(top, n, k, glu=glu, up_to=True)
    needs = [hab.linear_workspace_bytes(t, n, k, glu=glu) for t in range(top + 1)]
    assert most == max(needs)
    most = hab.sgmv_linear_workspace_bytes(p, top, n, k, 1, glu, up_to=True)
    needs = [hab.sgmv_linear_workspace_bytes(p, t, n, k, 1, glu) for t in range(top + 1)]
    assert most == max(needs)


def test_the_need_is_not_monotone():
    """Why one has to ask: a smaller batch may run in more parts."""
    needs = [hab.linear_workspace_bytes(t, 4096, 4096) for t in range(1, 513)]
    assert max(needs) > needs[-1]


def test_bad_requests():
    p = pool(4096, [4096])
    assert hab.linear_workspace_bytes(128, 4096, 4095, up_to=True) == 0
    assert hab.sgmv_linear_workspace_bytes(p, 128, 4096, 4096, 9, up_to=True) == 0
    other = hab.Plan(p, 64, [0, 64], [-1])
    assert hab.sgmv_linear_workspace_bytes(p, 128, 4096, 4096, 1, plan=other) == 0
    elsewhere = hab.Plan(pool(4096, [4096]), 128, [0, 128], [-1])
    assert hab.sgmv_linear_workspace_bytes(p, 128, 4096, 4096, 1, plan=elsewhere) == 0
    with pytest.raises(ValueError):
        hab.sgmv_linear_workspace_bytes(p, 64, 4096, 4096, 1, plan=other, up_to=True)
