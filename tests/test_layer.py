"""The operators around the delta, host side: refusals (nothing is enqueued,
so no GPU is needed)."""
import ctypes

import pytest

import heterogeneous_adapter_batching_amd as hab
from heterogeneous_adapter_batching_amd._lib import NormDesc

BF16, F32 = 1, 0
P = 1 << 30   # addresses that no call may reach


def norm_call(h=P, ldh=64, o=P + (1 << 20), ldo=64, post_w=0, post_b=0, gate=0, ldg=0, pre_w=0,
              pre_b=0, h_out=P + (2 << 20), ldho=64, u=P + (3 << 20), ldu=64, dtype=BF16,
              stream_dtype=BF16, T=4, width=64, post=0, pre=1, gate_act=0, unit=0, alpha=1.0,
              beta=1.0, eps=1e-5, desc=True):
    d = NormDesc(dtype, stream_dtype, T, width, post, pre, gate_act, unit, alpha, beta, eps)
    return hab.load().block_norm(ctypes.byref(d) if desc else None, h, ldh, o, ldo, post_w, post_b,
                                 gate, ldg, pre_w, pre_b, h_out, ldho, u, ldu, None)


EINVAL, EDTYPE = -1, -5


@pytest.mark.parametrize("bad, status", [
    (dict(desc=False), EINVAL), (dict(dtype=2), EDTYPE), (dict(stream_dtype=7), EDTYPE),
    (dict(dtype=F32, stream_dtype=BF16), EDTYPE), (dict(T=-1), EINVAL), (dict(width=0), EINVAL),
    (dict(width=32769, ldh=40000, ldo=40000, ldho=40000, ldu=40000), EINVAL),
    (dict(post=3), EINVAL), (dict(pre=-1), EINVAL), (dict(gate_act=3), EINVAL),
    (dict(unit=2), EINVAL), (dict(alpha=float("nan")), EINVAL), (dict(beta=float("inf")), EINVAL),
    (dict(eps=-1e-6), EINVAL), (dict(h=0), EINVAL), (dict(h=P + 1), EINVAL),
    (dict(u=P + (3 << 20) + 1), EINVAL), (dict(ldh=63), EINVAL), (dict(ldu=0), EINVAL),
    (dict(o=0, post=1), EINVAL), (dict(o=0, gate=P), EINVAL), (dict(post_w=P), EINVAL),
    (dict(pre=0), EINVAL), (dict(u=0), EINVAL), (dict(u=0, pre=0, h_out=0), EINVAL),
    (dict(u=P), EINVAL), (dict(h_out=P + 2), EINVAL), (dict(h_out=P, ldho=80), EINVAL),
    (dict(h_out=P + (1 << 20)), EINVAL), (dict(u=P + (2 << 20) + 64), EINVAL),
    (dict(gate=P + (3 << 20) + 2, ldg=64), EINVAL), (dict(pre_w=P + (3 << 20)), EINVAL),
    (dict(ldo=1 << 41), EINVAL),
])
def test_block_norm_refusals(bad, status):
    assert norm_call(**bad) == status
    assert hab.load().lora_last_error()


def test_block_norm_empty():
    """No tokens: the descriptor is checked, no tensor is."""
    assert norm_call(T=0, h=0, u=0, o=0) == 0
    assert norm_call(T=0, width=0) == EINVAL
