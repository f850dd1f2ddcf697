"""Arguments of the attention's calls at their borders, host side (nothing is
enqueued, so no GPU is needed)."""
import math

import pytest

from test_attention import EINVAL, ESTATE, M, P, attend, cache, rotary


@pytest.mark.parametrize("scale, status", [
    (3e38, EINVAL), (-3e38, EINVAL), (math.inf, EINVAL), (math.nan, EINVAL), (2.3e38, ESTATE),
    (-2.3e38, ESTATE), (0.0, ESTATE), (1e-45, ESTATE)])
def test_scales(scale, status):
    """A scale whose product with log2 e is past float32 would make 0 times
    infinity of scores of zero."""
    assert attend(scale=scale) == status


def layout(pages, heads, page, k, v, strides, vstrides=None):
    """rotary_append on a cache of such a layout (elements from its start), heads
    of 64."""
    c = cache(P + 2 * M + 2 * k, P + 2 * M + 2 * v, *strides, pages=pages)
    c.v_page_stride, c.v_head_stride, c.v_token_stride = vstrides or strides
    return rotary(c=c, heads=4 * heads, kv_heads=heads, page=page, ldq=16384, ldqo=256 * heads,
                  ldk=16384, ldv=16384, kv=True, per=64 // page + 1, ld_pages=64 // page + 1,
                  q=P, qo=P + M, k=P + 8192, v=P + 16384)


FAR = 1 << 24
LAYOUTS = [
    # (strides of pages, heads, tokens; where values start; whether places coincide)
    (dict(strides=(64, 2 ** 17, 64), v=FAR), True),          # page 1 token 0 is page 0 token 1
    (dict(strides=(2048, 64, 64), v=FAR), True),             # head 1 token 0 is head 0 token 1
    (dict(strides=(2048, 1024, 64), v=64), True),            # values a token on from the keys
    (dict(strides=(2048, 1024, 64), v=32), True),            # and half a token
    (dict(strides=(2048, 1024, 64), v=0), True),
    (dict(strides=(2048, 1024, 64), v=1024), True),          # head 0's values are head 1's keys
    (dict(strides=(2048, 1024, 64), v=2048), True),          # and the next page's
    (dict(strides=(1024, 1024, 64), v=FAR), True),
    (dict(strides=(2048, 960, 64), v=FAR), True),            # a head's last token is the next one's first
    (dict(strides=(2040, 1024, 64), v=FAR), True),           # the last elements of a page
    (dict(strides=(2048, 1024, 64), v=FAR), False),
    (dict(strides=(4096, 1024, 64), v=2048), False),         # a page's keys, then its values
    (dict(strides=(4096, 2048, 64), v=1024), False),         # a head's
    (dict(strides=(4096, 2048, 128), v=64), False),          # a token's
    (dict(strides=(4096, 128, 256), v=64), False),           # tokens ahead of heads, a head's two
    (dict(strides=(4096, 64, 256), v=128), False),           # a token's heads of keys, then of values
    (dict(strides=(4096, 64, 256), v=64), True),
    (dict(strides=(64, 64 * 200, 64 * 100), v=FAR), True),   # pages innermost: head 1 is token 2
    (dict(strides=(64, 64 * 100, 64 * 200), v=FAR), False),
    (dict(strides=(64, 64 * 1600, 64 * 100), v=FAR), False),
    (dict(strides=(128, 128 * 1600, 128 * 100), v=64), False),
    # no stride reaches past what the smaller ones span, and yet no two places meet
    (dict(strides=(320, 64 * 10001, 192), v=FAR, pages=3), False),
    (dict(strides=(320, 64 * 10001, 192), v=FAR, pages=4), True),
    # keys by heads and values by tokens
    (dict(strides=(4096, 1024, 64), vstrides=(4096, 64, 128), v=2048), False),
    (dict(strides=(4096, 1024, 64), vstrides=(4096, 64, 128), v=1984), True),
    (dict(strides=(4096, 1024, 64), vstrides=(4096, 64, 128), v=2112), True),
    (dict(strides=(4096, 1024, 64), vstrides=(2048, 64, 128), v=2048), True),
    (dict(strides=(2048, 1024, 64), vstrides=(2048, 64, 128), v=FAR), False),
    (dict(strides=(4096, 1024, 64), vstrides=(4096, 64, 128), v=2048 - 4096, k=4096), False),
]


@pytest.mark.parametrize("how, coincide", LAYOUTS)
def test_places_that_coincide_are_not_written(how, coincide):
    """Two places of the cache with elements in common would be written by two
    workgroups at once."""
    how = dict(dict(pages=100, heads=2, page=16, k=0), **how)
    how["v"] += how["k"]
    assert layout(**how) == (EINVAL if coincide else ESTATE)


def test_places_by_trying_every_pair():
    """Random small layouts against a count of every element's owners."""
    import random
    r = random.Random(5)
    seen = set()
    for _ in range(4000):
        pages, heads = r.choice([1, 2, 3, 5]), r.choice([1, 2, 3])
        step = r.choice([8, 64])
        strides = [step * r.randrange(1, r.choice([4, 20, 70, 140])) for _ in range(2)]
        strides.append(64 + step * r.randrange(0, r.choice([4, 20, 140])))
        v = step * r.randrange(0, r.choice([3, 30, 300, 900]))
        own, meets = set(), False
        for start in (0, v):
            for p in range(pages):
                for h in range(heads):
                    for t in range(16):
                        at = start + p * strides[0] + h * strides[1] + t * strides[2]
                        place = range(at, at + 64, 8)    # (everything is a multiple of 8 elements)
                        meets = meets or not own.isdisjoint(place)
                        own.update(place)
        got = layout(pages, heads, 16, 0, v, tuple(strides))
        assert got == (EINVAL if meets else ESTATE), (pages, heads, strides, v)
        seen.add((meets, pages > 1, heads > 1))
    assert len(seen) >= 7
