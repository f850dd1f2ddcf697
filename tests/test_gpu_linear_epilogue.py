"""The epilogue's activations where the exponential leaves float32's range."""
import pytest

from test_gpu_linear import BF16, F32, _gpu, act64  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [5, 40, 300])
def test_silu_far_left(T, dtype):
    """silu(v) = v e^v / (1 + e^v) is a normal number down to v = -91.  e^v by
    the hardware's base-2 exponential is off by |v| log2(e) 2^-24 < 2^-16.8
    relative for the argument's rounding, plus its own 2^-22; bf16 takes that
    one, float32 the library's, within 2 ulp; three more roundings.  Results
    under 2^-126 may be flushed."""
    import heterogeneous_adapter_batching_amd as hab
    x = torch.zeros(T, 64, dtype=dtype, device="cuda")
    x[:, 0] = torch.linspace(-104, -80, T).to(dtype)
    w = torch.zeros(72, 64, dtype=dtype, device="cuda")
    w[:, 0] = 1
    for act in ("silu", "gelu_tanh"):
        if act == "gelu_tanh":                       # z = 1.5958 (v + 0.044715 v^3) = -104 .. -80
            v = x[:, 0].double()
            u = torch.full_like(v, -10.0)
            for _ in range(60):
                f = 1.5957691216057308 * (u + 0.044715 * u ** 3) - v
                u = u - f / (1.5957691216057308 * (1 + 3 * 0.044715 * u ** 2))
            x[:, 0] = u.to(dtype)
        y = hab.frozen_linear(x, w, act=act)
        ref = act64(x[:, :1].double(), act).expand(T, 72)
        # gelu_tanh's z rounds four times (2^-22 of |z| <= 128 in the exponent)
        rel = torch.finfo(dtype).eps / 2 + (2.0 ** -16 if dtype == BF16 else 2.0 ** -20)
        if act == "gelu_tanh":
            rel += 2.0 ** -15
        bad = ((y.double() - ref).abs() / (rel * ref.abs() + 2.0 ** -126)).max().item()
        print(f"[linear] {act} {T} tokens {dtype}: {bad:.3f} of the bound", flush=True)
        assert bad <= 1.0
