"""A rebuild that runs out of host memory leaves the plan as it was (in a child
process with a limit on its memory; no GPU is used)."""
import os
import subprocess
import sys

from conftest import ROOT

RUN = r"""
import ctypes, resource, sys
import numpy as np
sys.path[:0] = [%r, %r]
import heterogeneous_adapter_batching_amd as hab
from test_attention import ESTATE, cache, ints

lib = hab.load()
plan = hab.AttentionPlan(8, 2, 64, 16, [5, 3], [9, 40])
before, size = plan.stats(), plan.workspace_bytes()
ones = np.ones(1 << 20, np.int32)
cases = ([1 << 22], [1 << 22]), (ones, 7 * ones)
now = next(int(l.split()[1]) << 10 for l in open("/proc/self/status") if l.startswith("VmSize"))
resource.setrlimit(resource.RLIMIT_AS, (now + (48 << 20), resource.RLIM_INFINITY))
for new, kv in cases:
    try:
        plan.rebuild(new, kv)
    except hab.LoraError as e:
        print(e)
    else:
        raise SystemExit("the rebuild found the memory")
    assert (plan.num_tokens, plan.num_seqs) == (8, 2)
    assert plan.stats() == before and plan.workspace_bytes() == size
    # (not uploaded: a call is refused, where a plan of no tokens succeeds)
    P = 1 << 32
    assert lib.paged_attention(plan.handle, P, 512, ctypes.byref(cache()), P << 1, 3, 3, 0.125,
                               P + (1 << 26), 512, None) == ESTATE
plan.rebuild([1], [2])
assert plan.stats()["tokens"] == plan.num_tokens == 1
print("all refused")
"""


def test_a_rebuild_without_memory():
    code = RUN % (ROOT, os.path.join(ROOT, "tests"))
    res = subprocess.run([sys.executable, "-c", code], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                         text=True, timeout=300, cwd=ROOT)
    assert res.returncode == 0 and "all refused" in res.stdout, res.stdout[-4000:]
