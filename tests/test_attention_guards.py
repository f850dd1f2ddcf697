"""The debug build's checks of the attention's tables, compiled for the host:
what they let through and what they hold back, at the borders and where sums of
32 bits would wrap (no GPU)."""
import os
import subprocess

from conftest import ROOT

CSRC = os.path.join(ROOT, "heterogeneous_adapter_batching_amd", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "attend_internal.h"
using namespace lora;
int main() {
    // 10 tokens of 3 sequences, 2 key heads of 4 query heads, 256 keys, 6 partial sums
    const AttnBounds b{10, 3, 2, 4, 256, 6, nullptr};
    const int32_t most = 0x7fffffff, least = -most - 1;
    const uint32_t T = kDbgToken, R = kDbgRow;
    // seq, kv_head, row0, rows, tok0, pos0, key0, key1, slot
    struct { AttnUnit u; uint32_t want; } units[] = {
        {{0, 0, 0, 40, 0, 0, 0, 256, -1}, 0}, {{2, 1, 16, 40, 0, 5, 192, 256, 5}, 0},
        {{-1, 99, -99, 99, 99, 99, 99, 99, 99}, 0}, {{1, 0, 0, 4, 9, -7, 64, 0, 0}, 0},
        {{0, 0, 40, 40, 0, most, 0, least, 0}, 0}, {{0, 0, 0, 37, 0, 0, 0, 1, 0}, 0},
        {{3, 0, 0, 4, 0, 0, 0, 1, 0}, R}, {{-2, 0, 0, 4, 0, 0, 0, 1, 0}, R},
        {{least, 0, 0, 4, 0, 0, 0, 1, 0}, R}, {{0, 2, 0, 4, 0, 0, 0, 1, 0}, T},
        {{0, -1, 0, 4, 0, 0, 0, 1, 0}, T}, {{0, 0, -16, 4, 0, 0, 0, 1, 0}, T},
        {{0, 0, 41, 40, 0, 0, 0, 1, 0}, T}, {{0, 0, 0, 41, 0, 0, 0, 1, 0}, T},
        {{0, 0, 0, 5, 9, 0, 0, 1, 0}, T}, {{0, 0, 0, 4, 10, 0, 0, 1, 0}, T},
        {{0, 0, 0, 4, -1, 0, 0, 1, 0}, T}, {{0, 0, 0, most, most, 0, 0, 1, 0}, T},
        {{0, 0, most, most, 0, 0, 0, 1, 0}, T}, {{0, 0, 0, -1, 0, 0, 0, 1, 0}, T},
        {{0, 0, 0, 4, 0, 0, -64, 1, 0}, R}, {{0, 0, 0, 4, 0, 0, 16, 64, 0}, R},
        {{0, 0, 0, 4, 0, 0, 0, 257, 0}, R}, {{0, 0, 0, 4, 0, 0, 0, most, 0}, R},
        {{0, 0, 0, 4, 0, 0, 0, 1, 6}, R}, {{0, 0, 0, 4, 0, 0, 0, 1, -2}, R},
        {{0, 0, 0, 4, 0, 0, 0, 1, most}, R}, {{3, 2, 0, 4, 0, 0, 0, 1, 0}, T | R}};
    // tok0, kv_head, row0, rows, slot0, slots
    struct { AttnJoin j; uint32_t want; } joins[] = {
        {{0, 0, 0, 40, 0, 6}, 0}, {{9, 1, 0, 4, 5, 1}, 0}, {{99, 99, -9, 99, 99, 0}, 0},
        {{0, 0, 0, 4, 1, 6}, R}, {{0, 0, 0, 4, 0, 7}, R}, {{0, 0, 0, 4, -1, 2}, R},
        {{0, 0, 0, 4, 2, -1}, R}, {{0, 0, 0, 4, most, most}, R}, {{0, 0, 0, 4, 1, most}, R},
        {{10, 0, 0, 4, 0, 2}, T}, {{0, 2, 0, 4, 0, 2}, T}, {{0, 0, 5, 4, 0, 2}, T}, {{0, 0, -1, 4, 0, 2}, T}};
    struct { AttnToken t; uint32_t want; } tokens[] = {
        {{0, 0}, 0}, {{2, 255}, 0}, {{1, -3}, 0}, {{1, least}, 0}, {{3, 0}, R}, {{-1, 0}, R}, {{0, 256}, R},
        {{0, most}, R}, {{most, 0}, R}};
    int bad = 0, n = 0;
    for (const auto &c : units) { ++n; if (wrong(b, c.u) != c.want) { std::printf("unit %d\n", n); ++bad; } }
    n = 0;
    for (const auto &c : joins) { ++n; if (wrong(b, c.j) != c.want) { std::printf("join %d\n", n); ++bad; } }
    n = 0;
    for (const auto &c : tokens) { ++n; if (wrong(b, c.t) != c.want) { std::printf("token %d\n", n); ++bad; } }
    const AttnBounds none{10, 3, 2, 4, 256, 0, nullptr};
    if (wrong(none, AttnUnit{0, 0, 0, 4, 0, 0, 0, 1, -1}) != 0) ++bad;
    if (wrong(none, AttnUnit{0, 0, 0, 4, 0, 0, 0, 1, 0}) != R) ++bad;
    std::printf("%d wrong\n", bad);
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


def test_table_entries_are_read_through_the_checks():
    """Every kernel checks the one entry that it reads."""
    for name, entry in (("attend.hip", "u"), ("attend_prompt.hip", "u"), ("attend.hip", "j"),
                        ("rotary.hip", "tok")):
        assert open(os.path.join(CSRC, name)).read().count(f"held(a.dbg, {entry})") == 1
    for name, reads in (("attend.hip", 2), ("attend_prompt.hip", 1), ("rotary.hip", 1)):
        text = open(os.path.join(CSRC, name)).read()
        assert sum(text.count(f"load_invariant(a.{t} +") for t in ("units", "joins", "tokens")) == reads
