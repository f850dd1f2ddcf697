"""block_norm on the GPU against its formula in 64 bits.

The tolerance of each element follows the formula's own rounding: u = 2^-24
for every float32 operation, L sequential additions at most in a row's sums
(32 values a lane in order, 4 DPP steps, 4 scalars, 16 waves: under 64 in
all), and half a step of the stored type for the one rounding at the end.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
L = 64
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import heterogeneous_adapter_batching_amd as hab
    hab.load()


def half_step(t, dtype):
    return torch.finfo(dtype).eps / 2 * t.abs()


def norm64(v, dv, kind, w, b, eps):
    """(value, error bound) of a norm of v known to dv, in 64 bits."""
    if kind == "none":
        return v, dv
    m, dm = 0.0, 0.0
    if kind == "layer":
        m = v.mean(1, keepdim=True)
        dm = (L + 1) * U * v.abs().mean(1, keepdim=True) + dv.mean(1, keepdim=True)
    t = v - m
    dt = dv + dm + U * t.abs()
    p = t.square().mean(1, keepdim=True)
    rt, rd = p.sqrt(), dt.square().mean(1, keepdim=True).sqrt()
    dp = p * (L + 3) * U + 2 * rt * rd + rd * rd
    f = 1.0 / torch.sqrt(p + eps)
    df = f * (0.5 * dp / (p + eps) + 4 * U)
    w = torch.ones_like(v[:1]) if w is None else w
    b = torch.zeros_like(v[:1]) if b is None else b
    r = t * f * w + b
    return r, dt * f * w.abs() + t.abs() * df * w.abs() + 4 * U * ((t * f * w).abs() + b.abs())


def reference(h, o, k):
    """(h_out, its bound, u, its bound) in 64 bits, on the CPU."""
    d = lambda t: None if t is None else t.detach().cpu().double()  # noqa: E731
    h = d(h)
    w = lambda t: None if t is None else d(t) + (1.0 if k.get("unit_offset") else 0.0)  # noqa: E731
    ho, dh = h * k.get("beta", 1.0), U * (h * k.get("beta", 1.0)).abs()
    if o is not None:
        n, dn = norm64(d(o), torch.zeros_like(h), k.get("post", "none"), w(k.get("post_weight")),
                       d(k.get("post_bias")), k.get("eps", 1e-5))
        if k.get("gate") is not None:
            g = d(k["gate"])
            g = {"none": lambda t: t, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[
                k.get("gate_act", "none")](g)
            dn = dn * g.abs() + 8 * U * (n * g).abs()
            n = n * g
        a = k.get("alpha", 1.0)
        ho = ho + a * n
        dh = dh + abs(a) * dn + 4 * U * ((a * n).abs() + h.abs() * abs(k.get("beta", 1.0)))
    if k.get("pre", "rms") == "none":
        return ho, dh, None, None
    u, du = norm64(ho, dh, k.get("pre", "rms"), w(k.get("pre_weight")), d(k.get("pre_bias")),
                   k.get("eps", 1e-5))
    return ho, dh, u, du


def check(h, o, k, got_h, got_u, what):
    ho, dh, u, du = reference(h, o, k)
    for name, got, ref, err in (("h_out", got_h, ho, dh), ("u", got_u, u, du)):
        if ref is None:
            assert got is None
            continue
        tol = err * 1.01 + half_step(ref.abs() + err, got.dtype) + 1e-37
        bad = ((got.cpu().double() - ref).abs() / tol).max().item() if ref.numel() else 0.0
        print(f"[norm] {what} {name}: {bad:.3f} of the bound", flush=True)
        assert bad <= 1.0, (what, name, bad)


def case(seed, T, d, dtype, stream, post, pre, gate, gate_act, bias):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0, mean=0.0, dt=dtype: (  # noqa: E731
        torch.randn(*s, generator=g) * std + mean).to(dt).cuda()
    h, o = r(T, d, std=2.0, mean=0.3, dt=stream), r(T, d, mean=-0.2)
    k = dict(post=post, pre=pre, gate_act=gate_act, alpha=0.37, beta=1.25)
    for side, kind in (("post", post), ("pre", pre)):
        if kind != "none":
            k[side + "_weight"] = r(d, std=0.1, mean=1.0)
            if bias:
                k[side + "_bias"] = r(d, std=0.1)
    if gate != "none":
        k["gate"] = r(d) if gate == "vector" else r(T, d)
    return h, o, k


WIDTHS = [1, 7, 8, 64, 100, 511, 513, 1024, 1030, 2048, 4096, 5003, 8192, 16384, 16392, 32768]


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, types):
    import heterogeneous_adapter_batching_amd as hab
    for i, (post, pre, gate, act, bias) in enumerate((
            ("none", "rms", "none", "none", False), ("rms", "rms", "vector", "none", False),
            ("layer", "layer", "rows", "tanh", True), ("rms", "none", "rows", "sigmoid", True))):
        h, o, k = case(width + i, 1 + 2 * i, width, *types, post, pre, gate, act, bias)
        got = hab.block_norm(h, o, **k)
        check(h, o, k, *got, f"{width} {types} {post}/{pre}/{gate}")


@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("T", [2, 5, 300, 4097])
def test_tokens(T, types):
    import heterogeneous_adapter_batching_amd as hab
    for d in (40, 320, 1000):
        h, o, k = case(T, T, d, *types, "layer", "rms", "rows", "sigmoid", True)
        check(h, o, k, *hab.block_norm(h, o, **k), f"T {T} d {d}")


def test_first_and_last_block():
    """No block output yet (the stream is returned as it is), a scaled copy,
    and the last update with no norm after it."""
    import heterogeneous_adapter_batching_amd as hab
    h, o, k = case(3, 33, 264, BF16, F32, "none", "rms", "none", "none", False)
    w = k["pre_weight"]
    ho, u = hab.block_norm(h, pre_weight=w)
    assert ho is h and u.dtype == BF16
    check(h, None, dict(pre_weight=w), h, u, "first")
    ho, u = hab.block_norm(h, pre_weight=w, beta=0.5)
    check(h, None, dict(pre_weight=w, beta=0.5), ho, u, "scaled")
    ho, u = hab.block_norm(h, o, pre="none", alpha=0.5)
    check(h, o, dict(pre="none", alpha=0.5), ho, u, "last")


def test_unit_offset_and_eps():
    import heterogeneous_adapter_batching_amd as hab
    h, o, k = case(4, 9, 520, F32, F32, "rms", "layer", "none", "none", True)
    k.update(unit_offset=True, eps=0.25)
    check(h, o, k, *hab.block_norm(h, o, **k), "unit offset")


def test_zero_rows_and_large_mean():
    """A row of zeros (its norm is the bias) and rows whose mean is far from
    their spread."""
    import heterogeneous_adapter_batching_amd as hab
    h, o, k = case(5, 6, 1000, F32, F32, "layer", "layer", "none", "none", True)
    h[0], o[0] = 0, 0
    h[1] += 1000.0
    o[2] += 4096.0
    check(h, o, k, *hab.block_norm(h, o, **k), "zeros and means")
    z = torch.zeros(2, 64, device="cuda")
    _, u = hab.block_norm(z, pre="layer", eps=1e-5)
    assert bool((u == 0).all())


def test_nan_and_inf_stay_in_their_rows():
    import heterogeneous_adapter_batching_amd as hab
    h, o, k = case(6, 8, 700, BF16, BF16, "rms", "rms", "vector", "none", False)
    clean = hab.block_norm(h, o, **k)
    h[2, 5], o[4, 699], o[7, 0] = float("nan"), float("inf"), float("-inf")
    ho, u = hab.block_norm(h, o, **k)
    rows = [0, 1, 3, 5, 6]
    assert torch.equal(ho[rows], clean[0][rows]) and torch.equal(u[rows], clean[1][rows])
    assert bool(u[[2, 4, 7]].isnan().all())


def test_strides_slices_and_in_place():
    """Rows at odd strides and offsets inside larger buffers, whose other
    elements stay as they were; h_out is h itself; rows behind the last."""
    import heterogeneous_adapter_batching_amd as hab
    T, d = 21, 333
    h, o, k = case(7, T, d, BF16, BF16, "rms", "layer", "rows", "tanh", True)
    want = hab.block_norm(h, o, **k)
    buf = torch.full((T + 4, 2 * d + 5), 7.0, dtype=BF16, device="cuda")
    hv, ov = buf[2:T + 2, 1:d + 1], buf[2:T + 2, d + 3:2 * d + 3]
    hv.copy_(h)
    ov.copy_(o)
    out = torch.full((T + 3, d + 9), 5.0, dtype=BF16, device="cuda")
    uv = out[1:T + 1, 3:d + 3]
    kk = dict(k, gate=torch.cat([k["gate"], k["gate"]], 1)[:, :d])
    ho, u = hab.block_norm(hv, ov, **kk, h_out=hv, u=uv)
    assert ho.data_ptr() == hv.data_ptr()
    assert torch.equal(hv, want[0]) and torch.equal(uv, want[1])
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[2:T + 2, 1:d + 1] = False
    keep[2:T + 2, d + 3:2 * d + 3] = False
    assert bool((buf[keep] == 7.0).all()) and torch.equal(ov, o)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:T + 1, 3:d + 3] = False
    assert bool((out[keep] == 5.0).all())


def test_far_rows():
    """Rows whose offsets pass 32 bits: 4200 rows 2^20 elements apart."""
    import heterogeneous_adapter_batching_amd as hab
    T, d, ld = 4200, 72, 1 << 20
    h, o, k = case(8, T, d, BF16, BF16, "none", "rms", "none", "none", False)
    want = hab.block_norm(h, o, **k)
    flat = torch.empty((T - 1) * ld + d, dtype=BF16, device="cuda")
    far = flat.as_strided((T, d), (ld, 1))
    far.copy_(h)
    ho, u = hab.block_norm(far, o, **k, h_out=far)
    assert torch.equal(far, want[0]) and torch.equal(u, want[1])


def test_graph_and_stream():
    """Captured on a stream of its own and replayed with new inputs."""
    import heterogeneous_adapter_batching_amd as hab
    h, o, k = case(9, 64, 1024, BF16, F32, "rms", "rms", "vector", "none", False)
    ho, u = torch.empty_like(h), torch.empty_like(o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        hab.block_norm(h, o, **k, h_out=ho, u=u)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        hab.block_norm(h, o, **k, h_out=ho, u=u)
    for seed in range(3):
        h2, o2, _ = case(20 + seed, 64, 1024, BF16, F32, "rms", "rms", "vector", "none", False)
        h.copy_(h2)
        o.copy_(o2)
        want = hab.block_norm(h, o, **k)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ho, want[0]) and torch.equal(u, want[1])


def test_empty_batch():
    import heterogeneous_adapter_batching_amd as hab
    h = torch.empty(0, 128, dtype=BF16, device="cuda")
    ho, u = hab.block_norm(h, h, pre="rms")
    assert ho.shape == u.shape == (0, 128)


def test_refused_tensors():
    import heterogeneous_adapter_batching_amd as hab
    h = torch.ones(4, 16, dtype=BF16, device="cuda")
    w = torch.ones(16, dtype=BF16, device="cuda")
    for bad, err in ((dict(o=h.cpu()), TypeError), (dict(o=h.float()), hab.LoraError),
                     (dict(o=h[:2]), ValueError), (dict(o=h, pre_weight=w[:8]), ValueError),
                     (dict(o=h, pre="max"), ValueError), (dict(o=h, gate_act="relu"), ValueError),
                     (dict(o=h, gate=w.float()), TypeError),
                     (dict(o=h, u=h), hab.LoraError), (dict(o=h.clone(), u=h), hab.LoraError),
                     (dict(o=h.clone(), h_out=h[:, :16].t().contiguous().t()), ValueError)):
        with pytest.raises(err):
            hab.block_norm(h, **bad)
    assert bool((h == 1).all())
