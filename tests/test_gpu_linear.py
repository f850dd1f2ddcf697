"""frozen_linear and sgmv_linear on the GPU against the formula in 64 bits.

Whole-number inputs make every product and sum exact in float32, whatever
the order, so those outputs must equal the reference's bits (one rounding to
bf16 at the end).  Real-valued inputs are held to the formula's own rounding:
u = 2^-24 for each of the at most k / 4 + 128 additions on a sum's path (a
matrix step adds at least 4 products; waves, splits and epilogue: under 128),
relative to the sum of the products' magnitudes, carried through the
activation by its slope, plus half a step of the stored type.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
NAMES = {BF16: "bf16", F32: "f32"}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import heterogeneous_adapter_batching_amd as hab
    hab.load()


def ints(g, *shape, top=2, dtype=BF16):
    return torch.randint(-top, top + 1, shape, generator=g).to(dtype).cuda()


def act64(v, act):
    return {"none": lambda: v, "relu": lambda: v.clamp(min=0), "silu": lambda: v * torch.sigmoid(v),
            "gelu": lambda: 0.5 * v * torch.erfc(-v / math.sqrt(2)),
            "gelu_tanh": lambda: v * torch.sigmoid(
                2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}[act]()


def end64(z, act, glu, residual):
    """act(z) [* up] + residual of float64 columns."""
    if glu:
        n = z.shape[1] // 2
        y = act64(z[:, :n], act) * z[:, n:]
    else:
        y = act64(z, act)
    return y if residual is None else y + residual.double()


# (T, k, n): one token to several tiles, odd widths, k inside and past one K
# tile, sizes that take each kernel, its split form and its edges
SIZES = [(1, 8, 1), (1, 264, 33), (3, 4096, 100), (16, 72, 1003), (17, 136, 64), (31, 1024, 48),
         (32, 2056, 31), (33, 8, 5), (40, 520, 300), (64, 4096, 128), (65, 1032, 257),
         (77, 1016, 1003), (128, 2048, 1024), (129, 200, 130), (200, 64, 4100), (256, 4096, 512),
         (300, 1048, 2050), (513, 328, 771), (700, 264, 6000), (1500, 136, 9000)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T, k, n", SIZES)
def test_exact_sizes(T, k, n, dtype):
    import heterogeneous_adapter_batching_amd as hab
    for glu, bias, res, act in ((False, False, False, "none"), (True, True, True, "relu"),
                                (False, True, True, "relu"), (True, False, False, "none")):
        g = torch.Generator().manual_seed(T * 7 + k + n)
        wide = 2 * n if glu else n
        x, w = ints(g, T, k, dtype=dtype), ints(g, wide, k, top=1, dtype=dtype)
        b = ints(g, wide, top=3, dtype=dtype) if bias else None
        r = ints(g, T, n, top=9, dtype=dtype) if res else None
        print(f"[linear] {T} x {k} x {n} {dtype} glu {glu} bias {bias} res {res}", flush=True)
        y = hab.frozen_linear(x, w, bias=b, act=act, glu=glu, residual=r)
        z = x.double() @ w.double().t()
        if b is not None:
            z = z + b.double()
        assert torch.equal(y, end64(z, act, glu, r).to(dtype)), (T, k, n, glu)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T, k, n", [(1, 1024, 200), (24, 1000, 129), (100, 2048, 260),
                                     (300, 1048, 2050), (1100, 520, 7000)])
def test_activations(T, k, n, act, dtype):
    import heterogeneous_adapter_batching_amd as hab
    g = torch.Generator().manual_seed(k + n)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype).cuda()  # noqa: E731
    for glu in (False, True):
        wide = 2 * n if glu else n
        x, w, b, res = r(T, k), r(wide, k, std=2 / math.sqrt(k)), r(wide), r(T, n)
        y = hab.frozen_linear(x, w, bias=b, act=act, glu=glu, residual=res)
        z = x.double() @ w.double().t() + b.double()
        mag = x.double().abs() @ w.double().abs().t() + b.double().abs()
        dz = (k / 4 + 128) * U * mag
        # the activations' slopes are at most 1.13; their own functions are
        # good to 2^-21 of |v| (float32) or 2^-19 (bf16's faster ones)
        fn = 2.0 ** -21 if dtype == F32 else 2.0 ** -19
        a = act64(z[:, :n], act)
        da = 1.13 * dz[:, :n] + fn * z[:, :n].abs()
        if glu:
            up, du = z[:, n:], dz[:, n:]
            ref, err = a * up, da * (up.abs() + du) + a.abs() * du + U * (a * up).abs()
        else:
            ref, err = a, da
        ref = ref + res.double()
        err = err + 2 * U * (ref.abs() + res.double().abs())
        tol = err + torch.finfo(dtype).eps / 2 * (ref.abs() + err)
        bad = ((y.double() - ref).abs() / tol).max().item()
        print(f"[linear] {T} x {k} x {n} {act} {dtype} glu {glu}: {bad:.3f} of the bound", flush=True)
        assert bad <= 1.0


def test_large_values_and_nan():
    """silu and gelu far from zero, relu and NaN; a NaN row of x stays in its
    row, a NaN row of w in its column."""
    import heterogeneous_adapter_batching_amd as hab
    for dtype in (BF16, F32):
        for T in (5, 40):
            x = torch.zeros(T, 64, dtype=dtype, device="cuda")
            x[:, 0] = torch.linspace(-200, 200, T).to(dtype)
            w = torch.zeros(72, 64, dtype=dtype, device="cuda")
            w[:, 0] = 1
            for act in ("silu", "gelu", "gelu_tanh", "relu"):
                y = hab.frozen_linear(x, w, act=act)
                ref = act64(x[:, :1].double(), act).expand(T, 72)
                tol = (torch.finfo(dtype).eps / 2 + 2.0 ** -18) * ref.abs() + 1e-30
                assert bool(((y.double() - ref).abs() <= tol).all()), (dtype, T, act)
            clean = hab.frozen_linear(x, w, act="relu")
            x[2], w[7] = float("nan"), float("nan")
            y = hab.frozen_linear(x, w, act="relu")
            assert bool(y[2].isnan().all()) and bool(y[:, 7].isnan().all())
            keep = torch.ones_like(y, dtype=torch.bool)
            keep[2], keep[:, 7] = False, False
            assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("T", [9, 30, 50, 100, 600])
def test_strides_slices_and_in_place(T):
    """x, w, residual and y as slices of larger buffers (y and residual at odd
    offsets and strides); y is the residual; rows behind the last stay."""
    import heterogeneous_adapter_batching_amd as hab
    g = torch.Generator().manual_seed(T)
    k, n = 200, 301
    xb, wb = ints(g, T + 2, k + 24), ints(g, n + 3, k + 40, top=1)
    xb[T + 1] = float("nan")
    wb[n + 2] = float("nan")
    x, w = xb[1:T + 1, 8:8 + k], wb[2:n + 2, 16:16 + k]
    out = ints(g, T + 4, n + 7, top=5)
    before = out.clone()
    y = out[2:T + 2, 3:n + 3]
    hab.frozen_linear(x, w, residual=y, y=y)
    ref = x.double() @ w.double().t() + before[2:T + 2, 3:n + 3].double()
    assert torch.equal(y, ref.to(BF16))
    before[2:T + 2, 3:n + 3] = y
    assert torch.equal(out, before)


def test_past_two_gib():
    """w of more than 2 GiB, and y of more than 2 GiB."""
    import heterogeneous_adapter_batching_amd as hab
    n, k = 140000, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(-1, 2, (n, k), generator=g, device="cuda", dtype=torch.int8).to(BF16)
    for T in (2, 70):
        x = torch.randint(-2, 3, (T, k), generator=g, device="cuda").to(BF16)
        y = hab.frozen_linear(x, w)
        at = torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")
        ref = x.double() @ w[at].double().t()
        assert torch.equal(y[:, at], ref.to(BF16)), T
    del w
    T, n, k = 9000, 130000, 64
    x = torch.randint(-2, 3, (T, k), generator=g, device="cuda").to(BF16)
    w = torch.randint(-2, 3, (n, k), generator=g, device="cuda").to(BF16)
    y = hab.frozen_linear(x, w)
    rows = torch.tensor([0, 4000, 8998, 8999], device="cuda")
    assert torch.equal(y[rows], (x[rows].double() @ w.double().t()).to(BF16))


@pytest.mark.parametrize("T", [4, 30, 90, 800])
def test_graph_and_stream(T):
    """Captured on a stream of its own and replayed with new inputs, with
    eager calls between the replays; deterministic."""
    import heterogeneous_adapter_batching_amd as hab
    g = torch.Generator().manual_seed(T)
    k, n = 1032, 520
    x, w = torch.randn(T, k, generator=g).to(BF16).cuda(), torch.randn(2 * n, k, generator=g).to(BF16).cuda()
    y = torch.empty(T, n, dtype=BF16, device="cuda")
    ws = torch.empty(max(1, hab.linear_workspace_bytes(T, n, k, "bf16", True)), dtype=torch.uint8,
                     device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        hab.frozen_linear(x, w, act="silu", glu=True, y=y, ws=ws)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        hab.frozen_linear(x, w, act="silu", glu=True, y=y, ws=ws)
    for i in range(3):
        x.copy_(torch.randn(T, k, generator=g).to(BF16))
        want = hab.frozen_linear(x, w, act="silu", glu=True)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    other = hab.frozen_linear(x, w, act="silu", glu=True, stream=s)
    s.synchronize()
    assert torch.equal(other, want)


# ------------------------------------------------------------ sgmv_linear ----

class Adapted:
    """A pool of whole-number adapters, a plan, and the delta in 64 bits."""

    def __init__(self, seed, T, k, widths, ranks, ids, starts, dtype=BF16, weights=None, layers=1,
                 skew=None, opts=None):
        import heterogeneous_adapter_batching_amd as hab
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.T, self.k, self.widths = dtype, T, k, widths
        self.starts, self.ids, self.weights = starts, ids, weights
        self.pool = hab.Pool(layers, [k] * len(widths), widths, r_max=64, dtype=NAMES[dtype],
                             slab_bytes=64 << 20)
        if opts:
            self.pool.set_plan_opts(**opts)
        self.ad = {}
        for i, r in enumerate(ranks):
            A = [ints(g, layers, r, k, top=1, dtype=dtype) for _ in widths]
            B = [ints(g, layers, w, r, top=1, dtype=dtype) for w in widths]
            scale = 0.5 * (1 + i % 3)
            self.ad[i] = (A, B, scale)
            self.pool.register(i, r, scale, A, B)
        self.plan = hab.Plan(self.pool, T, starts, ids, seg_weight=weights)
        self.plan.upload(max_proj=len(widths))

    def delta(self, x, layer, projs, offsets, wide):
        z = torch.zeros(self.T, wide, dtype=torch.float64, device="cuda")
        for s, i in enumerate(self.ids):
            lo, hi = int(self.starts[s]), int(self.starts[s + 1])
            if i < 0 or lo == hi:
                continue
            A, B, scale = self.ad[int(i)]
            wgt = 1.0 if self.weights is None else float(self.weights[s])
            for p, off in zip(projs, offsets):
                v = x[lo:hi].double() @ A[p][layer].double().t()
                z[lo:hi, off:off + self.widths[p]] += wgt * scale * (v @ B[p][layer].double().t())
        return z


def segments(seed, T, n_adapters, longest, idle=0.2):
    r = np.random.default_rng(seed)
    starts, ids = [0], []
    while starts[-1] < T:
        starts.append(min(T, starts[-1] + int(r.integers(0, longest + 1))))
        ids.append(-1 if r.random() < idle else int(r.integers(0, n_adapters)))
    return np.array(starts, np.int32), np.array(ids, np.int32)


def run_adapted(m, seed, n, offsets, projs=None, act="none", glu=False, bias=False, res=False,
                layer=0, what=""):
    import heterogeneous_adapter_batching_amd as hab
    g = torch.Generator().manual_seed(seed)
    projs = list(range(len(m.widths))) if projs is None else projs
    wide = 2 * n if glu else n
    x, w = ints(g, m.T, m.k, top=1, dtype=m.dtype), ints(g, wide, m.k, top=1, dtype=m.dtype)
    b = ints(g, wide, dtype=m.dtype) if bias else None
    r = ints(g, m.T, n, dtype=m.dtype) if res else None
    print(f"[adapted] {what} T {m.T} k {m.k} n {n} {m.dtype} glu {glu}", flush=True)
    y = hab.sgmv_linear(m.pool, m.plan, layer, projs, offsets, x, w, bias=b, act=act, glu=glu,
                        residual=r)
    z = x.double() @ w.double().t() + m.delta(x, layer, projs, offsets, wide)
    if b is not None:
        z = z + b.double()
    ref = end64(z, act, glu, r).to(m.dtype)
    bad = (y != ref).nonzero()
    assert bad.numel() == 0, (what, bad[:5].tolist(), len(bad))
    return x, w, y


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 5, 16, 29, 50, 100, 128, 200, 600])
def test_adapted_exact(T, dtype):
    """Ranks 3 to 64 mixed, short segments, tokens without an adapter."""
    ranks = [3, 8, 16, 13, 24, 32, 40, 64]
    starts, ids = segments(T, T, len(ranks), 9)
    m = Adapted(T, T, 264, [136, 72], ranks, ids, starts, dtype)
    run_adapted(m, T, 208, [0, 136], what="plain")
    run_adapted(m, T, 301, [100, 3], bias=True, res=True, act="relu", what="odd slices")
    m = Adapted(T + 1, T, 264, [136, 136], ranks, ids, starts, dtype)
    run_adapted(m, T, 136, [0, 136], glu=True, act="relu", bias=True, res=True, what="gated")
    m = Adapted(T + 1, T, 264, [272], ranks, ids, starts, dtype)
    run_adapted(m, T, 136, [0], glu=True, what="gated, one projection over both halves")


@pytest.mark.parametrize("T, n, k, longest", [(128, 4104, 1024, 1), (700, 6000, 136, 50),
                                              (1500, 9000, 72, 400), (1300, 520, 264, 300)])
def test_adapted_exact_larger(T, n, k, longest):
    starts, ids = segments(T, T, 5, longest)
    m = Adapted(T, T, k, [n], [8, 16, 64, 30, 64], ids, starts)
    run_adapted(m, T, n, [0], res=True, what="larger")
    m = Adapted(T, T, k, [n // 2 // 8 * 8] * 2, [8, 16, 64, 30, 64], ids, starts)
    run_adapted(m, T, n // 2 // 8 * 8, [0, n // 2 // 8 * 8], glu=True, what="larger, gated")


def test_adapted_long_groups():
    """A batch whose long groups take the prompt kernel's shrink, beside short ones."""
    T = 1400
    starts = np.array([0, 600, 601, 640, 1240, 1300, 1400], np.int32)
    ids = np.array([0, 1, -1, 2, 1, 0], np.int32)
    for dtype in (BF16, F32):
        m = Adapted(3, T, 136, [264, 64], [16, 8, 64], ids, starts, dtype)
        run_adapted(m, 3, 328, [0, 264], what="long groups")


@pytest.mark.parametrize("opts", [dict(long_group=1, long_batch=1), dict(long_group=6, long_batch=12),
                                  dict(long_group=10 ** 6), dict(shrink_groups=4096)])
@pytest.mark.parametrize("T", [7, 60, 300])
def test_adapted_plan_options(T, opts):
    """Plans whose groups are long or short by other thresholds, beside each
    other, at ranks of one K-step and more; many chunks of the shrink."""
    starts, ids = segments(T + 40, T, 4, 8)
    for ranks in ((8, 16, 24, 32), (8, 64, 48, 16)):
        for dtype in (BF16, F32):
            m = Adapted(T, T, 1032, [136, 72], ranks, ids, starts, dtype, opts=opts)
            run_adapted(m, T, 208, [0, 136], what=f"{opts}")


def test_adapted_many_projections():
    """Five projections in one call, short groups and long ones."""
    for T, longest in ((40, 3), (1400, 500)):
        starts, ids = segments(T, T, 3, longest)
        m = Adapted(T, T, 72, [8, 40, 16, 24, 64], [16, 8, 40], ids, starts)
        run_adapted(m, T, 152, [0, 8, 48, 64, 88], what="five projections")


def test_adapted_layers_weights_and_subsets():
    T = 90
    starts, ids = segments(8, T, 4, 5)
    wts = (np.random.default_rng(1).integers(-2, 3, len(ids)) * 0.5).astype(np.float32)
    m = Adapted(8, T, 72, [48, 40, 16], [8, 64, 20, 32], ids, starts, weights=wts, layers=3)
    run_adapted(m, 1, 104, [0, 48, 88], layer=2, what="weights, layer 2")
    run_adapted(m, 2, 56, [40, 0], projs=[2, 1], layer=1, what="two of three projections")


def test_adapted_none_and_empty():
    import heterogeneous_adapter_batching_amd as hab
    T = 20
    m = Adapted(9, T, 64, [64], [8], np.array([-1], np.int32), np.array([0, T], np.int32))
    x, w, y = run_adapted(m, 9, 64, [0], what="no adapters")
    assert torch.equal(y, hab.frozen_linear(x, w))
    m = Adapted(9, 0, 64, [64], [8], np.array([], np.int32), np.array([0], np.int32))
    assert hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], x[:0], w).shape == (0, 64)


def test_adapted_equals_two_steps():
    """In float32 against frozen_linear followed by sgmv_fused in place: the
    same sums, each rounded a few times (real values)."""
    import heterogeneous_adapter_batching_amd as hab
    g = torch.Generator().manual_seed(5)
    T, k, n = 70, 512, 264
    starts, ids = segments(5, T, 4, 6)
    m = Adapted(5, T, k, [n], [8, 16, 64, 32], ids, starts, F32)
    x, w = torch.randn(T, k, generator=g).cuda(), torch.randn(n, k, generator=g).cuda()
    y = hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], x, w)
    two = hab.frozen_linear(x, w)
    hab.sgmv_fused(m.pool, m.plan, 0, [0], [0], x, two)
    mag = x.abs() @ w.abs().t() + 1.5 * 64 * (x.abs().sum(1, keepdim=True))
    assert bool(((y - two).abs() <= (k / 4 + 256) * U * mag).all())


def test_adapted_nan_stays_with_its_adapter():
    """An adapter with NaN weights touches its own tokens alone, beside others
    in the same 16-token tile."""
    import heterogeneous_adapter_batching_amd as hab
    T = 48
    ids = np.arange(T, dtype=np.int32) % 3
    m = Adapted(6, T, 64, [64], [8, 64, 16], ids, np.arange(T + 1, dtype=np.int32))
    x, w, clean = run_adapted(m, 6, 64, [0], what="clean")
    A, B, s = m.ad[1]
    for bad in (float("nan"), float("inf")):
        m.pool.upload(1, 0, 0, A[0][0], torch.full_like(B[0][0], bad))
        y = hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], x, w)
        rows = torch.from_numpy(ids != 1).cuda()
        assert torch.equal(y[rows], clean[rows])
        assert not bool(y[~rows].isfinite().any(1).all())


def test_adapted_rebuild_graph_and_repeat():
    """A rebuilt plan over the same workspace; captured and replayed; the
    same bits every time."""
    import heterogeneous_adapter_batching_amd as hab
    T = 64
    starts, ids = segments(3, T, 4, 4)
    m = Adapted(3, T, 264, [136], [8, 16, 64, 32], ids, starts)
    run_adapted(m, 1, 136, [0], what="first")
    starts, ids = segments(4, T, 4, 3)
    m.plan.rebuild(T, starts, ids).upload(1, ws=torch.empty_like(m.plan.ws) if
                                          m.plan.workspace_bytes(1) <= m.plan.ws.numel() else None)
    m.starts, m.ids = starts, ids
    x, w, y = run_adapted(m, 2, 136, [0], what="rebuilt")
    out = torch.empty_like(y)
    ws = torch.empty(hab.sgmv_linear_workspace_bytes(m.pool, T, 136, 264, 1), dtype=torch.uint8,
                     device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], x, w, y=out, ws=ws)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], x, w, y=out, ws=ws)
    for i in range(3):
        x.copy_(torch.randn_like(x))
        want = hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], x, w)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refused_calls():
    import heterogeneous_adapter_batching_amd as hab
    T = 40
    starts, ids = segments(3, T, 2, 4)
    m = Adapted(3, T, 64, [64], [8, 16], ids, starts)
    x, w, y = run_adapted(m, 1, 64, [0])
    call = lambda **k: hab.sgmv_linear(  # noqa: E731
        m.pool, k.pop("plan", m.plan), k.pop("layer", 0), [0], k.pop("off", [0]),
        k.pop("x", x), k.pop("w", w), **k)
    merge = hab.Plan.merge(m.pool, T, [0, T], [[0, 1]], [[1.0, 1.0]]).upload(1)
    cores = hab.Plan(m.pool, T, [0, T], [0], seg_sigma=[0]).upload(1)
    fresh = hab.Plan(m.pool, T, [0, T], [0])
    for bad, err in ((dict(plan=merge), hab.LoraError), (dict(plan=cores), hab.LoraError),
                     (dict(plan=fresh), hab.LoraError), (dict(layer=1), hab.LoraError),
                     (dict(off=[1]), hab.LoraError), (dict(off=[-1]), hab.LoraError),
                     (dict(off=[0, 0]), ValueError), (dict(x=x[:8]), hab.LoraError),
                     (dict(x=x.float(), w=w.float()), hab.LoraError), (dict(w=w.float()), TypeError),
                     (dict(w=w[:, :56]), ValueError), (dict(glu=True, w=w[:63]), ValueError),
                     (dict(ws=torch.empty(256, dtype=torch.uint8, device="cuda")), hab.LoraError),
                     (dict(ws=m.plan.ws), hab.LoraError), (dict(y=x), hab.LoraError), (dict(act="sin"), ValueError),
                     (dict(residual=x[:, :63]), ValueError)):
        with pytest.raises(err):
            call(**bad)
    assert torch.equal(call(), y)


def test_sequence_of_a_decoder_layer():
    """The operators as a decoder layer runs them around its attention (here
    the identity on the value columns), captured into one graph and replayed
    on new inputs: norms, the adapted q/k/v, o onto the stream through the
    next norms, the gated MLP and its down projection.  Every stage is held to
    its formula in 64 bits on the inputs the run gave it."""
    import heterogeneous_adapter_batching_amd as hab
    from test_gpu_norm import check as check_norm
    h, kv, ffn, T = 512, 128, 1032, 150
    dt = BF16
    starts, ids = segments(11, T, 5, 9)
    g = torch.Generator().manual_seed(11)
    r = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).to(dt).cuda()  # noqa: E731
    shapes = {"q": (h, h), "k": (h, kv), "v": (h, kv), "o": (kv, h), "gate": (h, ffn),
              "up": (h, ffn), "down": (ffn, h)}
    pool = hab.Pool(1, [s[0] for s in shapes.values()], [s[1] for s in shapes.values()], 64,
                    "bf16", slab_bytes=32 << 20)
    ads = {}
    for a, rank in enumerate((8, 16, 64, 24, 40)):
        A = [r(1, rank, k, std=1 / math.sqrt(3 * k)) for k, _ in shapes.values()]
        B = [r(1, n, rank, std=0.05) for _, n in shapes.values()]
        ads[a] = (A, B)
        pool.register(a, rank, 2.0, A, B)
    plan = hab.Plan(pool, T, starts, ids).upload(max_proj=3)
    w = {"qkv": r(h + 2 * kv, h, std=1 / math.sqrt(h)), "o": r(h, kv, std=1 / math.sqrt(kv)),
         "gu": r(2 * ffn, h, std=1 / math.sqrt(h)), "down": r(h, ffn, std=1 / math.sqrt(ffn))}
    n1, n2, n3, post, gate = (r(h, std=0.1, mean=1.0) for _ in range(5))
    stream, first = r(T, h), {}

    def layer():
        s = {}
        _, s["x1"] = hab.block_norm(stream, pre_weight=n1)
        s["qkv"] = hab.sgmv_linear(pool, plan, 0, (0, 1, 2), (0, h, h + kv), s["x1"], w["qkv"])
        s["val"] = s["qkv"][:, h + kv:]
        s["att"] = hab.sgmv_linear(pool, plan, 0, (3,), (0,), s["val"], w["o"])
        s["h1"], s["x2"] = hab.block_norm(stream, s["att"], post="rms", post_weight=post, gate=gate,
                                          alpha=0.7, pre_weight=n2)
        s["mid"] = hab.sgmv_linear(pool, plan, 0, (4, 5), (0, ffn), s["x2"], w["gu"], act="silu",
                                   glu=True)
        s["h2"] = hab.sgmv_linear(pool, plan, 0, (6,), (0,), s["mid"], w["down"], residual=s["h1"])
        _, s["x3"] = hab.block_norm(s["h2"], pre="layer", pre_weight=n3)
        return s

    def delta(x, wide, projs, offs):
        z = torch.zeros(T, wide, dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(z)
        for s, i in enumerate(ids):
            lo, hi = int(starts[s]), int(starts[s + 1])
            if i < 0:
                continue
            for p, off in zip(projs, offs):
                A, B = (m[p][0].double() for m in ads[int(i)])
                n = B.shape[0]
                z[lo:hi, off:off + n] += 2 * (x[lo:hi].double() @ A.t()) @ B.t()
                mag[lo:hi, off:off + n] += 2 * (x[lo:hi].double().abs() @ A.abs().t()) @ B.abs().t()
        return z, mag

    def check_product(what, got, x, wt, projs, offs, act="none", glu=False, residual=None):
        k = x.shape[1]
        d, dmag = delta(x, wt.shape[0], projs, offs)
        z = x.double() @ wt.double().t() + d
        dz = (k / 4 + 256) * U * (x.double().abs() @ wt.double().abs().t() + dmag)
        ref = end64(z, act, glu, residual)
        if glu:
            n = z.shape[1] // 2
            a = act64(z[:, :n], act)
            da = 1.13 * dz[:, :n] + 2.0 ** -19 * z[:, :n].abs()
            err = da * (z[:, n:].abs() + dz[:, n:]) + a.abs() * dz[:, n:] + U * (a * z[:, n:]).abs()
        else:
            err = dz
        if residual is not None:
            err = err + 2 * U * (ref.abs() + residual.double().abs())
        bad = ((got.double() - ref).abs() / (err + torch.finfo(dt).eps / 2 * (ref.abs() + err))).max()
        print(f"[layer] {what}: {bad.item():.3f} of the bound", flush=True)
        assert bad <= 1.0, what

    def check_all(s):
        check_norm(stream, None, dict(pre_weight=n1), stream, s["x1"], "first norm")
        check_product("qkv", s["qkv"], s["x1"], w["qkv"], (0, 1, 2), (0, h, h + kv))
        check_product("o", s["att"], s["val"], w["o"], (3,), (0,))
        check_norm(stream, s["att"], dict(post="rms", post_weight=post, gate=gate, alpha=0.7,
                                          pre_weight=n2), s["h1"], s["x2"], "both norms")
        check_product("gate and up", s["mid"], s["x2"], w["gu"], (4, 5), (0, ffn), "silu", True)
        check_product("down", s["h2"], s["mid"], w["down"], (6,), (0,), residual=s["h1"])
        check_norm(s["h2"], None, dict(pre="layer", pre_weight=n3), s["h2"], s["x3"], "last norm")

    first = layer()
    check_all(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = layer()
    for _ in range(3):
        stream.copy_(r(T, h))
        eager = layer()
        graph.replay()
        torch.cuda.synchronize()
        for name in out:
            assert torch.equal(out[name], eager[name]), name
    check_all(out)


def test_two_streams_at_once():
    """Products and norms on two streams at once, each with its own plan and
    workspaces, give the bits of the calls alone."""
    import heterogeneous_adapter_batching_amd as hab
    T = 96
    runs = []
    for seed in (21, 22):
        starts, ids = segments(seed, T, 4, 3)
        m = Adapted(seed, T, 520, [264], [8, 16, 64, 32], ids, starts)
        g = torch.Generator().manual_seed(seed)
        x, w = torch.randn(T, 520, generator=g).to(BF16).cuda(), torch.randn(264, 520, generator=g).to(BF16).cuda()
        want = hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], x, w, act="silu")
        runs.append((m, x, w, want, torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for _ in range(20):
        for m, x, w, _, s, got in runs:
            got.append(hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], x, w, act="silu", stream=s))
    torch.cuda.synchronize()
    for _, _, _, want, _, got in runs:
        assert all(torch.equal(y, want) for y in got)


def test_rows_behind_a_padded_batch():
    """A batch padded to a captured size: rows without a segment of their own
    take no adapter, and the rows behind num_tokens are left alone."""
    import heterogeneous_adapter_batching_amd as hab
    T, pad = 37, 64
    starts, ids = segments(31, T, 3, 4)
    m = Adapted(31, T, 136, [72], [8, 24, 64], ids, starts)
    g = torch.Generator().manual_seed(3)
    xb, w = ints(g, pad, 136, top=1), ints(g, 72, 136, top=1)
    yb = torch.full((pad, 72), 3.0, dtype=BF16, device="cuda")
    hab.sgmv_linear(m.pool, m.plan, 0, [0], [0], xb[:T], w, y=yb[:T])
    assert bool((yb[T:] == 3.0).all())
    padded = hab.Plan(m.pool, pad, np.append(starts, pad), np.append(ids, -1)).upload(1)
    y = hab.sgmv_linear(m.pool, padded, 0, [0], [0], xb, w)
    assert torch.equal(y[:T], yb[:T])
    assert torch.equal(y[T:], (xb[T:].double() @ w.double().t()).to(BF16))


@pytest.mark.parametrize("rmax, granule", [(8, 8), (16, 16), (48, 16)])
def test_adapted_pool_shapes(rmax, granule):
    """Pools of other largest ranks and rank granules."""
    import heterogeneous_adapter_batching_amd as hab
    for dtype in (BF16, F32):
        g = torch.Generator().manual_seed(rmax)
        T, k, n = 30, 72, 40
        pool = hab.Pool(2, [k, 64], [n, 8], rmax, NAMES[dtype], rank_granule=granule, slab_bytes=4 << 20)
        ads = []
        for a, rank in enumerate((1, rmax // 2, rmax)):
            A = [ints(g, 2, rank, i, top=1, dtype=dtype) for i in (k, 64)]
            B = [ints(g, 2, o, rank, top=1, dtype=dtype) for o in (n, 8)]
            pool.register(a, rank, 1.0, A, B)
            ads.append((A, B))
        ids = np.arange(T, dtype=np.int32) % 4 - 1
        plan = hab.Plan(pool, T, np.arange(T + 1, dtype=np.int32), ids).upload(1)
        x, w = ints(g, T, k, top=1, dtype=dtype), ints(g, n + 5, k, top=1, dtype=dtype)
        y = hab.sgmv_linear(pool, plan, 1, [0], [5], x, w)
        z = x.double() @ w.double().t()
        for t, a in enumerate(ids):
            if a >= 0:
                z[t, 5:] += (x[t].double() @ ads[a][0][0][1].double().t()) @ ads[a][1][0][1].double().t()
        assert torch.equal(y, z.to(dtype))
