"""What the package gives on a machine without torch (no GPU)."""
import os
import subprocess
import sys

from conftest import ROOT


def run(code):
    return subprocess.run([sys.executable, "-c", "import sys; sys.modules['torch'] = None\n" + code],
                          cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT), stdout=subprocess.PIPE,
                          stderr=subprocess.STDOUT, text=True, timeout=120)


def test_every_name_of_the_package():
    res = run("from heterogeneous_adapter_batching_amd import *\n"
              "import heterogeneous_adapter_batching_amd as hab\n"
              "assert all(n in globals() for n in hab.__all__), hab.__all__\n"
              "print(linear_workspace_bytes(128, 4096, 14336))")
    assert res.returncode == 0, res.stdout
    assert int(res.stdout) > 0


def test_a_plan_and_its_workspaces():
    """Sizes need no torch: a planner asks for them on a machine of its own."""
    res = run("import heterogeneous_adapter_batching_amd as hab\n"
              "p = hab.Pool(1, [4096], [4096], r_max=16, slab_ptr=1 << 30, slab_bytes=1 << 30)\n"
              "p.reserve(0, 16, 1.0)\n"
              "plan = hab.Plan(p, 64, [0, 32, 64], [0, -1])\n"
              "print(hab.sgmv_linear_workspace_bytes(p, 64, 4096, 4096, 1, plan=plan))")
    assert res.returncode == 0, res.stdout
    assert int(res.stdout) > 0


def test_the_operators_themselves_refuse():
    res = run("import heterogeneous_adapter_batching_amd as hab\n"
              "try:\n"
              "    hab.block_norm([1.0])\n"
              "except TypeError as e:\n"
              "    print('refused:', e)")
    assert res.returncode == 0 and "refused: h must be a CUDA tensor" in res.stdout, res.stdout
