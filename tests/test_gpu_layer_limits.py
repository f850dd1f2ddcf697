"""On the GPU: more rows than one launch of the norms holds."""
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
