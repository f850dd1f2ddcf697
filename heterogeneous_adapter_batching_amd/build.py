"""Build the gfx950 library libhab_lora.so in-tree with hipcc.

The library is the C ABI of include/lora_sgmv.h: host code (pool, plan,
validation) and the HIP kernels, linked into one shared object that the
Python binding loads with ctypes.
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libhab_lora.so")
# the same library with the kernels' bounds checks compiled in (LORA_SGMV_DEBUG)
DEBUG_LIB = os.path.join(PKG, "libhab_lora_debug.so")
DEBUG_FLAGS = ["-DLORA_SGMV_DEBUG"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = [os.path.join(CSRC, "lora_sgmv.cpp"), os.path.join(CSRC, "exchange.cpp"),
           os.path.join(CSRC, "layer.cpp"), os.path.join(CSRC, "kernels.hip"),
           os.path.join(CSRC, "norm.hip"), os.path.join(CSRC, "linear.hip"),
           os.path.join(CSRC, "attend.cpp"), os.path.join(CSRC, "attend.hip"),
           os.path.join(CSRC, "attend_prompt.hip"), os.path.join(CSRC, "rotary.hip")]

# Packed float32 ALU ops are switched off for all device code; the compiler's
# host pass warns that it does not know the feature, which is harmless.
FLAGS = ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC",
         "-Wall", "-Wextra", "-Wno-unused-parameter",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", INCLUDE, "-I", CSRC]


def _run(cmd) -> None:
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    noise = "is not a recognized feature for this target"
    log = "\n".join(l for l in res.stdout.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{log}")
    if log.strip():
        print(log, file=sys.stderr)


def _build_many(jobs) -> list:
    """Builds [(out, extra flags)], every source of every library compiled
    side by side, then linked."""
    with tempfile.TemporaryDirectory(dir=PKG, prefix=".build_") as tmp, \
            ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
        objs = [[os.path.join(tmp, f"{n}_{os.path.basename(s)}.o") for s in SOURCES]
                for n in range(len(jobs))]
        # the largest translation units first
        work = sorted(((os.path.getsize(s), s, o, extra)
                       for (_, extra), os_ in zip(jobs, objs) for s, o in zip(SOURCES, os_)),
                      key=lambda t: -t[0])
        for f in [pool.submit(_run, [HIPCC, *FLAGS, *extra, "-c", s, "-o", o])
                  for _, s, o, extra in work]:
            f.result()
        for (out, extra), os_ in zip(jobs, objs):
            _run([HIPCC, f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", out + ".tmp", *os_])
            os.replace(out + ".tmp", out)
    return [out for out, _ in jobs]


def build(out: str = LIB, extra=()) -> str:
    return _build_many([(out, list(extra))])[0]


def build_all() -> list:
    """The library and its debug build."""
    return _build_many([(LIB, []), (DEBUG_LIB, DEBUG_FLAGS)])


# The host sources built with g++ alone (no device code: host_only.cpp
# stands in for the kernel launchers) under AddressSanitizer and
# UndefinedBehaviorSanitizer, to run the host-side tests against.
SANITIZE = ["-fsanitize=address,undefined", "-fno-omit-frame-pointer", "-fno-sanitize-recover=all"]


def host_sanitized(out: str) -> str:
    srcs = [os.path.join(CSRC, "lora_sgmv.cpp"), os.path.join(CSRC, "exchange.cpp"),
            os.path.join(CSRC, "layer.cpp"), os.path.join(CSRC, "attend.cpp"),
            os.path.join(CSRC, "host_only.cpp")]
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", *SANITIZE,
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", INCLUDE, "-I", CSRC, *srcs,
           "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", out]
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed ({res.returncode}):\n{res.stdout}")
    return out


if __name__ == "__main__":
    print(build_all())
