"""Infinities and NaN of one adapter's weights in sgmv_linear on the GPU: the
delta is added on its projection's slice and nowhere else, and an infinite
weight gives what the formula gives.

The expected values are the formula's in 64 bits, whose infinities and NaN
are IEEE's own: finite outputs come from whole numbers and must equal the
reference's bits; the others must be the same infinity, or NaN where it is.
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


def same(got, ref):
    return (got == ref) | (got.isnan() & ref.isnan())


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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T, k, wide, seg, ranks", SIZES)
def test_infinite_b(T, k, wide, seg, ranks, dtype):
    """Single infinities and NaN in B: s v_r times the infinity, NaN only where
    v_r is zero, where infinities of both signs meet, or where B is NaN."""
    import heterogeneous_adapter_batching_amd as hab
    m, offsets, token = make(T, k, wide, seg, ranks, dtype, False)
    g = torch.Generator().manual_seed(T + 1)
    x, w = ints(g, T, k, top=1, dtype=dtype), ints(g, wide, k, top=1, dtype=dtype)
    A, B, _ = m.ad[1]
    for p in (0, 1):
        Bp = B[p][0]
        Bp[2, 0], Bp[5, -1], Bp[m.widths[p] - 1, 1] = INF, -INF, INF
        Bp[9, 0], Bp[9, 2] = INF, -INF
        Bp[11, 3] = NAN
        m.pool.upload(1, 0, p, A[p][0], Bp)
    y = hab.sgmv_linear(m.pool, m.plan, 0, [0, 1], offsets, x, w)
    z = (x.double() @ w.double().t()).cpu()
    token, xc = token.cpu(), x.double().cpu()
    for a, (A, B, s) in m.ad.items():
        rows = token == a
        for p, off in enumerate(offsets):
            v = s * (xc[rows] @ A[p][0].double().cpu().t())
            z[rows, off:off + m.widths[p]] += (v[:, None, :] * B[p][0].double().cpu()[None]).sum(2) \
                if a == 1 and T < 1000 else v @ B[p][0].double().cpu().t()
    ref = z.to(dtype).cuda()
    print(f"[nonfinite] {T} x {k} x {wide} ranks {ranks} {dtype}: {int(ref.isinf().sum())} infinities, "
          f"{int(ref.isnan().sum())} NaN", flush=True)
    assert bool(ref.isinf().any()) and bool(ref.isnan().any())
    bad = (~same(y, ref)).nonzero()
    assert bad.numel() == 0, (bad[:5].tolist(), len(bad))


def test_infinite_b_of_real_values():
    """The same where v fills all three bf16 pieces: the sign of v decides."""
    import heterogeneous_adapter_batching_amd as hab
    for T, k, wide, seg, ranks in SIZES:
        m, offsets, token = make(T, k, wide, seg, ranks, BF16, False)
        g = torch.Generator().manual_seed(T + 2)
        x = torch.randn(T, k, generator=g).to(BF16).cuda()
        w = torch.randn(wide, k, generator=g).to(BF16).cuda()
        A, B, s = m.ad[1]
        B[0][0][4, 1], B[0][0][7, -1] = INF, -INF
        m.pool.upload(1, 0, 0, A[0][0], B[0][0])
        y = hab.sgmv_linear(m.pool, m.plan, 0, [0, 1], offsets, x, w)
        rows = token == 1
        v = s * (x[rows].double() @ A[0][0].double().t())
        print(f"[nonfinite] real values, {T} x {k} x {wide} ranks {ranks}", flush=True)
        assert torch.equal(y[rows][:, offsets[0] + 4].double(), v[:, 1] * INF)
        assert torch.equal(y[rows][:, offsets[0] + 7].double(), v[:, -1] * -INF)
        y[rows.nonzero()[:, 0, None], torch.tensor([[offsets[0] + 4, offsets[0] + 7]], device="cuda")] = 0
        assert bool(y.isfinite().all())
