"""Arguments of the attention's calls at their borders, host side (nothing is
enqueued, so no GPU is needed)."""
import math

import pytest

from test_attention import EINVAL, ESTATE, attend


@pytest.mark.parametrize("scale, status", [
    (3e38, EINVAL), (-3e38, EINVAL), (math.inf, EINVAL), (math.nan, EINVAL), (2.3e38, ESTATE),
    (-2.3e38, ESTATE), (0.0, ESTATE), (1e-45, ESTATE)])
def test_scales(scale, status):
    """A scale whose product with log2 e is past float32 would make 0 times
    infinity of scores of zero."""
    assert attend(scale=scale) == status
