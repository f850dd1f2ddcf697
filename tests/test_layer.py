"""The operators around the delta, host side: refusals (nothing is enqueued,
so no GPU is needed)."""
import ctypes

import pytest

import heterogeneous_adapter_batching_amd as hab
from heterogeneous_adapter_batching_amd._lib import LinearDesc, NormDesc

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


def linear_call(x=P, ldx=64, w=P + (1 << 24), ldw=64, bias=0, residual=0, ldr=40, y=P + (2 << 24),
                ldy=40, ws=P + (3 << 24), ws_bytes=1 << 24, dtype=BF16, T=4, n=40, k=64, act=0,
                glu=0, desc=True):
    d = LinearDesc(dtype, T, n, k, act, glu)
    return hab.load().frozen_linear(ctypes.byref(d) if desc else None, x, ldx, w, ldw, bias,
                                    residual, ldr, y, ldy, ws, ws_bytes, None)


@pytest.mark.parametrize("bad, status", [
    (dict(desc=False), EINVAL), (dict(dtype=3), EDTYPE), (dict(T=-1), EINVAL), (dict(n=0), EINVAL),
    (dict(k=0), EINVAL), (dict(k=60), EINVAL), (dict(k=1 << 21, ldx=1 << 21, ldw=1 << 21), EINVAL),
    (dict(act=5), EINVAL), (dict(act=-1), EINVAL), (dict(glu=2), EINVAL),
    (dict(T=1 << 30, n=1 << 20), EINVAL), (dict(x=0), EINVAL), (dict(x=P + 8), EINVAL),
    (dict(ldx=56), EINVAL), (dict(ldx=68), EINVAL), (dict(ldw=1 << 21), EINVAL),
    (dict(w=0), EINVAL), (dict(w=P + (1 << 24) + 2), EINVAL), (dict(y=0), EINVAL),
    (dict(y=P + (2 << 24) + 1), EINVAL), (dict(ldy=39), EINVAL), (dict(ldr=39, residual=P), EINVAL),
    (dict(bias=P + 1), EINVAL), (dict(y=P), EINVAL), (dict(y=P + (1 << 24) + 64), EINVAL),
    (dict(bias=P + (2 << 24)), EINVAL), (dict(residual=P + (2 << 24) + 2), EINVAL),
    (dict(residual=P + (2 << 24), ldr=48), EINVAL),
    (dict(T=100, k=4096, ldx=4096, ldw=4096, ws=0), EINVAL),
    (dict(T=100, k=4096, ldx=4096, ldw=4096, ws=P + (3 << 24) + 16), EINVAL),
    (dict(T=100, k=4096, ldx=4096, ldw=4096, ws_bytes=64), -9),
    (dict(T=100, k=4096, ldx=4096, ldw=4096, ws=P + (2 << 24)), EINVAL),
])
def test_frozen_linear_refusals(bad, status):
    assert linear_call(**bad) == status
    assert hab.load().lora_last_error()


def test_frozen_linear_empty():
    assert linear_call(T=0, x=0, w=0, y=0, ws=0) == 0
    assert linear_call(T=0, k=3) == EINVAL


def test_linear_workspace_bytes():
    """No workspace for one token or for products with tiles enough; a bound by
    the sizes alone otherwise; 0 for a bad descriptor."""
    assert hab.linear_workspace_bytes(1, 4096, 4096) == 0
    assert hab.linear_workspace_bytes(4096, 14336, 4096, glu=True) == 0
    n = hab.linear_workspace_bytes(128, 4096, 14336)
    assert n % 256 == 0 and 4 * 128 * 4096 * 2 <= n <= 4 * 128 * 4224 * 64
    assert hab.linear_workspace_bytes(128, 4096, 14337) == 0
    pool = hab.Pool(1, [4096], [4096], r_max=64, slab_ptr=1 << 20, slab_bytes=1 << 24)
    assert hab.sgmv_linear_workspace_bytes(pool, 128, 4096, 4096, 1) == \
        hab.linear_workspace_bytes(128, 4096, 4096) + (4 + 6) * 128 * 64
    assert hab.sgmv_linear_workspace_bytes(pool, 128, 4096, 4096, 0) == 0


def test_sgmv_linear_host_refusals():
    """What needs no device: an unuploaded plan, another pool's plan."""
    pool = hab.Pool(1, [64], [64], r_max=64, slab_ptr=1 << 20, slab_bytes=1 << 24)
    plan = hab.Plan(pool, 4, [0, 4], [-1])
    lib, one = hab.load(), (ctypes.c_int32 * 1)(0)
    d = LinearDesc(BF16, 4, 64, 64, 0, 0)
    args = (0, 1, one, one, ctypes.byref(d), P, 64, P + (1 << 20), 64, None, None, 64,
            P + (2 << 20), 64, None, 0, None)
    assert lib.sgmv_linear(pool.handle, plan.handle, *args) == -9
    assert lib.sgmv_linear(None, plan.handle, *args) == EINVAL
