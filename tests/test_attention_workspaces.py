"""Workspaces that plans of both kinds are uploaded into, in turn and in part
over one another: a call whose tables are no longer there is refused, and so is
one whose tensors reach into them (host side, no GPU)."""
import host_library

RUN = r"""
import ctypes
import numpy as np
import heterogeneous_adapter_batching_amd as hab
from heterogeneous_adapter_batching_amd._lib import RotaryDesc
from test_attention import M, P, cache

EINVAL, ESTATE, EHIP = -1, -9, -7
lib = hab.load()
pool = hab.Pool(1, [64], [64], 8, "bf16", slab_ptr=P, slab_bytes=1 << 20)

memory = np.zeros(1 << 20, np.uint8)
base = -(-memory.ctypes.data // 256) * 256


def attention(new=(1, 4), kv=(9, 40)):
    return hab.AttentionPlan(8, 2, 64, 16, list(new), list(kv))


def adapters(T=8):
    return hab.Plan(pool, T, [0, T], [-1])


def upload(plan, at):
    if isinstance(plan, hab.Plan):
        n = lib.lora_plan_workspace_bytes(plan.handle, 1)
        assert lib.lora_plan_upload(plan.handle, at, n, 1, None) == 0
    else:
        n = plan.workspace_bytes()
        assert lib.attn_plan_upload(plan.handle, at, n, None) == 0
    return n


def call(plan, q=P, o=P + M, c=None, ldq=512, ldo=512):
    if isinstance(plan, hab.Plan):
        one, zero = (ctypes.c_int32 * 1)(0), (ctypes.c_int32 * 1)(0)
        return lib.sgmv_fused(pool.handle, plan.handle, 0, 1, one, zero, P, 64, None, 0, P + M, 64, None)
    return lib.paged_attention(plan.handle, q, ldq, ctypes.byref(c or cache()), P + 4 * M, 3, 3, 0.125, o,
                               ldo, None)


def rotary(plan, q=P, qo=P + M, k=P + 1024, v=P + 1280, c=None):
    d = RotaryDesc(64, 0, 1.0)
    return lib.rotary_append(plan.handle, ctypes.byref(d), q, 768, qo, 512, k, 768, v, 768,
                             ctypes.byref(c or cache()), P + 4 * M, 3, 3, None, P + 5 * M, None)


def held(plan):
    st = call(plan)
    assert st in (ESTATE, EHIP) or isinstance(plan, hab.Plan) and st == 0, st
    return st != ESTATE


# each kind over each, at the same place and part of the way
for first in (attention, adapters):
    for second in (attention, adapters):
        for shift in (0, 256, -256, "end", "front"):
            a, b = first(), second()
            at = base + 65536
            assert not held(a)
            n = upload(a, at)
            assert held(a)
            m = b.workspace_bytes() if isinstance(b, hab.AttentionPlan) else \
                lib.lora_plan_workspace_bytes(b.handle, 1)
            to = at + (-(-n // 256) * 256 if shift == "end" else -(-m // 256) * -256 if shift == "front" else shift)
            apart = to >= at + n or to + m <= at
            upload(b, to)
            assert held(b) and held(a) == apart, (first, second, shift)
            if not apart:
                upload(a, at)                    # and the other way round
                assert held(a) and not held(b)
            b.close()
            assert held(a)
            a.close()

# one plan uploaded twice, to places that overlap
a = attention()
upload(a, base)
upload(a, base + 256)
assert held(a)
upload(b := adapters(), base)
assert held(b) and held(a) == (lib.lora_plan_workspace_bytes(b.handle, 1) <= 256)
a, b = attention(), adapters()

# tensors and caches that reach into the workspace
n = upload(a, base)
inside = base + n - 16
assert call(a) == EHIP and rotary(a) == EHIP
assert call(a, o=inside) == EINVAL and call(a, q=inside) == EINVAL
assert call(a, o=base + n) == EHIP and call(a, q=base + n) == EHIP
assert call(a, c=cache(k=inside)) == EINVAL and call(a, c=cache(v=inside)) == EINVAL
for name in ("q", "qo", "k", "v"):
    assert rotary(a, **{name: inside}) == EINVAL, name
assert rotary(a, c=cache(k=inside)) == EINVAL and rotary(a, c=cache(v=inside)) == EINVAL
print("all held")
"""


def test_workspaces_of_both_kinds(tmp_path):
    assert "all held" in host_library.run(tmp_path, RUN)
