"""The library's host sources built with host_hip.cpp in place of the HIP
runtime, for tests of uploads and checks that run in a child process without a
GPU: there every call whose arguments hold ends with LORA_EHIP, at its launch."""
import glob
import os
import subprocess
import sys

from conftest import ROOT
from heterogeneous_adapter_batching_amd import build


def run(tmp_path, code):
    """Runs Python `code` with that library, and returns what it printed."""
    out = str(tmp_path / "libhab_lora_host.so")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-Wl,-z,defs",
                    "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", build.INCLUDE, "-I", build.CSRC,
                    *sorted(glob.glob(os.path.join(build.CSRC, "*.cpp"))),
                    os.path.join(here, "host_hip.cpp"), "-o", out], check=True)
    res = subprocess.run([sys.executable, "-c", code], env=dict(
        os.environ, HAB_LORA_LIB=out, PYTHONPATH=os.pathsep.join([ROOT, here])), cwd=ROOT,
        stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)
    assert res.returncode == 0, res.stdout[-4000:]
    return res.stdout
