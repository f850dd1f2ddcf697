"""Infinities and NaN of one adapter's weights in sgmv_linear on the GPU: the
delta is added on its projection's slice and nowhere else.
"""
import numpy as np
import pytest

from test_gpu_linear import BF16, F32, Adapted, _gpu, ints, segments  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")
# a few tokens; a product in parts with a join (ranks of one K-step and more);
# one launch with the delta's own K tiles, and the same with several ranks
SIZES = [(6, 256, 320, 1, (8, 16, 24)), (6, 256, 320, 1, (40, 64, 8)),
         (100, 2048, 320, 1, (16, 8, 24)), (100, 2048, 320, 1, (64, 40, 8)),
         (2048, 64, 4096, 512, (16, 16, 8)), (2048, 64, 4096, 512, (64, 40, 8))]


def make(T, k, wide, seg, ranks, dtype, glu):
    """Two projections whose slices start and end inside tiles, with columns
    of no projection before, between and behind them."""
    starts = np.minimum(np.arange(0, T + seg, seg), T).astype(np.int32)
    ids = (np.arange(len(starts) - 1, dtype=np.int32) % 4) - 1
    widths = [wide // 4 // 8 * 8 + 8, wide // 3 // 8 * 8 + 8]
    offsets = [3, wide // 2 - 5] if not glu else [5, wide // 2 + 9]
    m = Adapted(T + wide, T, k, widths, list(ranks), ids, starts, dtype)
    return m, offsets, torch.from_numpy(np.repeat(ids, np.diff(starts))).cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("T, k, wide, seg, ranks", SIZES)
def test_other_columns_are_left_alone(T, k, wide, seg, ranks, glu, dtype):
    """A of one adapter's first projection is not finite: its tokens' outputs
    in that slice are NaN, every other output keeps its bits."""
    import heterogeneous_adapter_batching_amd as hab
    m, offsets, token = make(T, k, wide, seg, ranks, dtype, glu)
    g = torch.Generator().manual_seed(T)
    x, w = ints(g, T, k, top=1, dtype=dtype), ints(g, wide, k, top=1, dtype=dtype)
    n = wide // 2 if glu else wide
    call = lambda: hab.sgmv_linear(m.pool, m.plan, 0, [0, 1], offsets, x, w, glu=glu)  # noqa: E731
    clean = call()
    assert bool(clean.isfinite().all())
    cols = torch.zeros(wide, dtype=torch.bool, device="cuda")
    cols[offsets[0]:offsets[0] + m.widths[0]] = True
    if glu:                               # gate and up of an output
        cols = cols[:n] | cols[n:]
    hit = (token == 1)[:, None] & cols[None, :]
    A, B, _ = m.ad[1]
    for bad in (NAN, INF):
        m.pool.upload(1, 0, 0, torch.full_like(A[0][0], bad), B[0][0])
        print(f"[nonfinite] {T} x {k} x {wide} ranks {ranks} glu {glu} {dtype} A {bad}", flush=True)
        y = call()
        moved = (y != clean) & ~hit
        assert not bool(moved.any()), moved.nonzero()[:5].tolist()
        assert not bool(y[hit].isfinite().any())
