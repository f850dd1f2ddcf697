"""The debug build's checks of every table entry that the product with adapters
reads, in a process of its own (this one has the release build loaded)."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_debug_build_checks_the_products_tables():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from heterogeneous_adapter_batching_amd import build
    assert os.path.exists(build.DEBUG_LIB), "build the library first (__graft_entry__.build())"
    run = os.path.join(ROOT, "tests", "debug_product_tables_run.py")
    print(f"[debug] {run} with the debug build", flush=True)
    res = subprocess.run([sys.executable, "-u", run], env=dict(os.environ, HAB_LORA_LIB=build.DEBUG_LIB),
                         cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                         timeout=100)
    print(res.stdout[-4000:], flush=True)
    assert res.returncode == 0, res.stdout[-4000:]
    assert "[debug] all checks passed" in res.stdout
