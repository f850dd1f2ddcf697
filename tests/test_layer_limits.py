"""Products and norms at the ends of their sizes, host side (addresses that no
call may reach; nothing is enqueued)."""
import ctypes

import pytest

import heterogeneous_adapter_batching_amd as hab
from heterogeneous_adapter_batching_amd._lib import LinearDesc

BF16, F32 = 1, 0
EINVAL = -1
GIB = 1 << 30


def linear(T, n, k=8, dtype=BF16, glu=0):
    d = LinearDesc(dtype, T, n, k, 0, glu)
    at = [GIB * 4096 * i for i in range(1, 5)]           # 4 TiB apart
    return hab.load().frozen_linear(ctypes.byref(d), at[0], k, at[1], k, 0, 0, 0, at[2], n, at[3],
                                    GIB * 4096, None)


@pytest.mark.parametrize("T, n, dtype, glu", [
    (2, 1 << 28, BF16, 0), (12, 1 << 28, F32, 0), (1, 1 << 28, BF16, 1),    # rows of W, 16 a workgroup
    (2 ** 31 - 1, 1, BF16, 0), (2 ** 31 - 256, 1, BF16, 0), (2 ** 31 - 1, 64, F32, 0),
    (1 << 30, 1, F32, 0), ((1 << 30) + 1, 8, F32, 1)])                      # token tiles of 32
def test_more_than_a_launch_holds_is_refused(T, n, dtype, glu):
    """A launch holds fewer than 2^32 threads, and token rows are counted in
    32 bits with a tile's length to spare."""
    assert linear(T, n, dtype=dtype, glu=glu) == EINVAL
    assert b"launch" in hab.load().lora_last_error() or b"num_tokens" in hab.load().lora_last_error()


def test_sizes_at_the_end():
    """The workspace queries take them without overflow."""
    for T in (2 ** 31 - 1, 2 ** 31 - 300, 2 ** 31 - 1024):
        assert hab.linear_workspace_bytes(T, 1, 8) >= 0
