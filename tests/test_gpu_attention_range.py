"""Attention where float32's range ends, and rows whose bits follow their own
keys alone."""
import pytest
import torch

from attention_reference import Batch
from test_gpu_attention import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seed", [0, 1])
def test_rows_follow_the_keys_that_they_see(seed, dim):
    """Keys that only later tokens of a chunk see, small or large, change no
    bit of the earlier ones' results."""
    seqs, at = 128, 64 + 26                      # (tokens of one wave see it, or do not)
    b = Batch([64] * seqs, [128] * seqs, heads=16, kv_heads=16, dim=dim, page=64, seed=seed)
    first = run(b)
    pages = b.pages[:, at // b.page].long()
    b.k[pages, :, at % b.page] *= 30
    other = run(b)
    sees = torch.cat([b.seen(s)[:, at] for s in range(seqs)])
    assert torch.equal(first[~sees], other[~sees])
    assert not torch.equal(first[sees], other[sees])
