"""float32 rows of 4097 to 8192: few of them and many take different numbers of
waves a row; each is held to the formula in 64 bits at the borders."""
import pytest

from test_gpu_norm import F32, _gpu, case, check  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T", [1, 512, 513, 1021])
@pytest.mark.parametrize("width", [4097, 5003, 5120, 5121, 8185])
def test_borders(T, width):
    import heterogeneous_adapter_batching_amd as hab
    for i, (post, pre, gate, bias) in enumerate((("none", "rms", "none", False),
                                                 ("layer", "layer", "rows", True))):
        h, o, k = case(T + width + i, T, width, F32, F32, post, pre, gate, "tanh", bias)
        check(h, o, k, *hab.block_norm(h, o, **k), f"{T} x {width} {post}/{pre}")
