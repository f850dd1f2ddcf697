"""The debug build's checks, compiled for the host: what they let through and
what they hold back, at the borders and where sums of 32 or 64 bits would
wrap (no GPU)."""
import os
import subprocess

from conftest import ROOT

CSRC = os.path.join(ROOT, "heterogeneous_adapter_batching_amd", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "sgmv_internal.h"
using namespace lora;
int main() {
    const DebugBounds d{1000, 40, 48};
    const int32_t most = 0x7fffffff, least = -most - 1;
    const uint64_t top = ~0ull;
    struct { const char *what; bool got, want; } t[] = {
        {"block 0 + 1000", block_inside(d, 0, 1000), true},
        {"block 1000 + 0", block_inside(d, 1000, 0), true},
        {"block 1 + 1000", block_inside(d, 1, 1000), false},
        {"block 1001 + 0", block_inside(d, 1001, 0), false},
        {"block top + 2", block_inside(d, top, 2), false},
        {"block 2 + top", block_inside(d, 2, top), false},
        {"block top - 499 + 1000", block_inside(d, top - 499, 1000), false},
        {"token -1", token_inside(d, -1), true}, {"token 0", token_inside(d, 0), true},
        {"token 39", token_inside(d, 39), true}, {"token 40", token_inside(d, 40), false},
        {"token -2", token_inside(d, -2), false}, {"token most", token_inside(d, most), false},
        {"token least", token_inside(d, least), false},
        {"rows 0 + 48", rows_inside(d, 0, 48), true}, {"rows 48 + 0", rows_inside(d, 48, 0), true},
        {"rows 1 + 48", rows_inside(d, 1, 48), false}, {"rows -1 + 2", rows_inside(d, -1, 2), false},
        {"rows 2 + -1", rows_inside(d, 2, -1), false},
        {"rows most + 1", rows_inside(d, most, 1), false},
        {"rows 1 + most", rows_inside(d, 1, most), false},
        {"rows most + most", rows_inside(d, most, most), false},
        {"group 0 of 3", group_inside(3, 0), true}, {"group 2 of 3", group_inside(3, 2), true},
        {"group 3 of 3", group_inside(3, 3), false}, {"group -1 of 3", group_inside(3, -1), false},
        {"group 0 of 0", group_inside(0, 0), false},
        {"rank 8", padded_rank(8), true}, {"rank 64", padded_rank(64), true},
        {"rank 0", padded_rank(0), false}, {"rank 12", padded_rank(12), false},
        {"rank 72", padded_rank(72), false}, {"rank -8", padded_rank(-8), false},
        {"rank 1 << 20", padded_rank(1 << 20), false}};
    int bad = 0;
    for (const auto &c : t)
        if (c.got != c.want) { std::printf("%s: %d\n", c.what, c.got); ++bad; }
    std::printf("%d checks, %d wrong\n", int(sizeof t / sizeof *t), bad);
    return bad != 0;
}
"""


def test_guards(tmp_path):
    src, exe = tmp_path / "guards.cpp", tmp_path / "guards"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", CSRC,
                    "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert res.returncode == 0, res.stdout


def test_plan_rows_are_read_through_the_checks():
    """The product's kernels read token rows and adapter blocks in one place
    each, where the debug build checks them."""
    text = open(os.path.join(CSRC, "linear.hip")).read()
    assert text.count(".order[") == 1 and text.count("token_row(") == 5
    assert text.count("slab_bytes") == 0 and text.count("block_bytes(") == 3
