"""Attention where float32's range ends: values near its largest, scales of
zero and next to it; and rows whose bits follow their own keys alone."""
import math

import pytest
import torch

from attention_reference import Batch
from test_gpu_attention import check, run

pytestmark = pytest.mark.gpu


def place(b, s, j):
    return int(b.pages[s, j // b.page]), j % b.page


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new, kv", [(32, 200), (130, 400), (40, 9000)])
def test_values_near_the_largest(new, kv, dim):
    """A key that scores 2^7.8 times the earlier ones' weights, whose value is
    2^122: a running maximum left where it was would bring its product to
    2^129.8, and the row to infinity."""
    b = Batch([new], [kv], heads=4, kv_heads=2, dim=dim, seed=kv)
    b.q.zero_()
    b.q.view(b.tokens, 4, dim)[..., 0] = 8.0
    b.k.copy_(torch.where(b.k.isnan(), b.k, torch.zeros_like(b.k)))
    page, slot = place(b, 0, 150)
    b.k[page, :, slot, 0] = 5.4375               # score 5.4375: 2^7.845
    b.v[page, :, slot] = b.v[page, :, slot].sign() * 2.0 ** 122
    check(b, run(b, scale=0.125), 0.125)


def test_values_near_the_largest_beside_infinite_ones():
    """The same where a later value, which the last tokens alone see, is
    infinite: theirs is, the others' are right."""
    b = Batch([64], [260], heads=2, kv_heads=2, seed=1)
    b.q.zero_()
    b.q.view(b.tokens, 2, b.dim)[..., 0] = 8.0
    b.k.copy_(torch.where(b.k.isnan(), b.k, torch.zeros_like(b.k)))
    page, slot = place(b, 0, 150)
    b.k[page, :, slot, 0] = 5.4375
    b.v[page, :, slot] = b.v[page, :, slot].sign() * 2.0 ** 122
    clean = run(b, scale=0.125)
    check(b, clean, 0.125)
    page, slot = place(b, 0, 250)
    b.v[page, :, slot, 3] = math.inf
    o = run(b, scale=0.125)
    sees = b.seen(0)[:, 250]
    assert torch.equal(o[~sees], clean[~sees]) and sees.any() and (~sees).any()
    o, clean = (t.view(b.tokens, 2, b.dim) for t in (o, clean))
    assert (o[sees][..., 3] == math.inf).all()
    o[..., 3], clean[..., 3] = 0, 0
    assert torch.equal(o, clean)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("scale", [0.0, 1e-36, -1e-36, 1e-38, 2e-40])
def test_scales_next_to_zero(scale, new, dtype):
    """Products of 10^36 and more, brought into range (or to nothing) by the
    scale."""
    b = Batch([new], [300], dtype=dtype, seed=3)
    b.q.mul_(1e18)
    b.k.mul_(1e18)
    check(b, run(b, scale=scale), scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 60])
def test_a_scale_of_zero_and_infinite_products(new, dtype):
    """0 times an infinite product is no number."""
    b = Batch([new], [300], dtype=dtype, seed=4)
    b.k[place(b, 0, 7)[0], :, place(b, 0, 7)[1], 5] = math.inf
    assert run(b, scale=0.0).isnan().all()


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
