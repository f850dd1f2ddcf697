"""The attention's host code (plans, validation) under AddressSanitizer and
UndefinedBehaviorSanitizer: its host tests against a build without device code,
in a child process.  No GPU is used."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT
from heterogeneous_adapter_batching_amd import build as lib_build


def test_plans_under_sanitizers(tmp_path):
    asan = subprocess.run(["g++", "-print-file-name=libasan.so"], stdout=subprocess.PIPE,
                          text=True).stdout.strip()
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("no libasan for g++")
    env = dict(os.environ, HAB_LORA_LIB=lib_build.host_sanitized(str(tmp_path / "libhab_lora_san.so")),
               LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                          os.path.join(ROOT, "tests", "test_attention.py")],
                         cwd=ROOT, env=env, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                         timeout=600)
    tail = "\n".join(res.stdout.splitlines()[-40:])
    assert res.returncode == 0 and " passed" in tail, tail
    assert "ERROR: AddressSanitizer" not in res.stdout and "runtime error:" not in res.stdout, tail
