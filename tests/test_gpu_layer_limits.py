"""On the GPU: more rows than one launch of the norms holds, and the widest
product of a few tokens that one launch holds."""
import pytest

from test_gpu_linear import BF16, F32, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T, width, stream", [((1 << 26) + 3, 2, BF16), ((1 << 23) + 5, 8, F32),
                                              (1 << 23, 3, BF16)])
def test_norm_of_more_rows_than_a_launch(T, width, stream):
    """Whole-number rows: the stream's update is exact, and the RMS norm of a
    row of equal magnitudes m is +-m / sqrt(m^2 + eps)."""
    import heterogeneous_adapter_batching_amd as hab
    print(f"[norm] {T} x {width}", flush=True)
    i = torch.arange(T, device="cuda")
    h = ((i % 13) - 6).to(stream)[:, None].repeat(1, width)
    o = ((i % 7) + 1).to(BF16)[:, None].repeat(1, width)
    gate = ((i % 3) + 1).to(BF16)[:, None].repeat(1, width)
    ho, u = hab.block_norm(h, o, gate=gate, pre="rms", eps=1.0)
    want = h.float() + o.float() * gate.float()
    assert torch.equal(ho, want.to(stream))
    ref = want / torch.sqrt(want * want + 1.0)
    assert bool(((u.float() - ref).abs() <= (2.0 ** -8 + 2.0 ** -20) * ref.abs()).all())


def test_widest_product_of_two_tokens():
    import heterogeneous_adapter_batching_amd as hab
    n = (1 << 28) - 4096
    print(f"[linear] 2 x 8 x {n}", flush=True)
    w = torch.ones(n, 8, dtype=BF16, device="cuda")
    w[::3, 1] = -2
    x = torch.tensor([[1, 2, 0, 0, 1, 0, 0, 3], [0, 1, 1, 0, 0, 0, 2, 0]], dtype=BF16, device="cuda")
    y = hab.frozen_linear(x, w)
    for t, (other, third) in enumerate(((7.0, 1.0), (4.0, 1.0))):
        assert bool((y[t, ::3] == third).all())
        assert bool((y[t, 1::3] == other).all()) and bool((y[t, 2::3] == other).all())
