"""Descriptors of the operators around the delta, host side: the values a call
is given are the values the library gets."""
import ctypes

import pytest

import heterogeneous_adapter_batching_amd as hab
import heterogeneous_adapter_batching_amd.layer as layer
from heterogeneous_adapter_batching_amd._lib import NormDesc

torch = pytest.importorskip("torch")


def test_scales_given_as_tensors_are_read_at_each_call(monkeypatch):
    """A scale held in a tensor (a layer's parameter) is read when the call is
    made, not remembered by the tensor it came in."""
    seen = []
    monkeypatch.setattr(layer, "_matrix", lambda t, *a: (0, t.shape[1]))
    monkeypatch.setattr(layer, "_enqueue", lambda fn, args, *a: seen.append(
        ctypes.cast(args[0], ctypes.POINTER(NormDesc)).contents))
    h, o = torch.zeros(4, 64), torch.zeros(4, 64)
    alpha, beta, eps = torch.tensor(0.5), torch.tensor(1.5), torch.tensor(0.25)
    for k in (1.0, 2.0, 8.0):
        hab.block_norm(h, o, alpha=alpha, beta=beta, eps=eps, h_out=h, u=o)
        assert (seen[-1].alpha, seen[-1].beta, seen[-1].eps) == (0.5 * k, 1.5 * k, 0.25 * k)
        for t in (alpha, beta, eps):
            t.mul_(2.0 if k == 1.0 else 4.0)
    a = torch.tensor(2.0)
    for k in (2.0, 5.0):                      # one of them alone
        hab.block_norm(h, o, alpha=a, h_out=h, u=o)
        assert seen[-1].alpha == k
        a.fill_(5.0)


def test_scales_that_are_no_numbers_are_refused(monkeypatch):
    monkeypatch.setattr(layer, "_matrix", lambda t, *a: (0, t.shape[1]))
    monkeypatch.setattr(layer, "_enqueue", lambda *a: pytest.fail("enqueued"))
    h = torch.zeros(4, 64)
    for bad in (None, "1", torch.zeros(2), [1.0]):
        for name in ("alpha", "beta", "eps"):
            with pytest.raises((TypeError, ValueError, RuntimeError)):
                hab.block_norm(h, h, u=h, h_out=h, **{name: bad})


BIG = (1 << 32) + 4          # 4, if only 32 bits of it were kept


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """The C structures hold 32 bits, and ctypes drops the others."""
    pool = hab.Pool(1, [64], [64], r_max=64, slab_ptr=1 << 20, slab_bytes=1 << 24)
    for call in (lambda: hab.linear_workspace_bytes(BIG, 4096, 4096),
                 lambda: hab.linear_workspace_bytes(128, BIG, 4096),
                 lambda: hab.linear_workspace_bytes(128, 4096, BIG + 4),
                 lambda: hab.sgmv_linear_workspace_bytes(pool, BIG, 64, 64, 1),
                 lambda: hab.sgmv_linear_workspace_bytes(pool, 128, 64, 64, BIG - 3),
                 lambda: hab.api._offsets([BIG]), lambda: hab.api._projs([BIG])):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    monkeypatch.setattr(layer, "_matrix", lambda t, *a: (0, t.shape[1]))
    monkeypatch.setattr(layer, "_enqueue", lambda *a: pytest.fail("enqueued"))
    row = torch.zeros(1, 8, dtype=torch.bfloat16)
    tall = row.expand(BIG, 8)
    with pytest.raises(ValueError, match="32 bits"):
        hab.block_norm(tall, h_out=tall, u=tall)
    with pytest.raises(ValueError, match="32 bits"):
        hab.frozen_linear(tall, row, y=tall)
    with pytest.raises(ValueError, match="32 bits"):
        hab.frozen_linear(row, tall, y=tall)
    plan = hab.Plan(pool, 1, [0, 1], [-1])
    with pytest.raises(ValueError, match="32 bits"):
        hab.sgmv_linear(pool, plan, BIG - 4, [0], [0], row, row, y=row)
