"""The pairs of bf16 parts whose products stand for an fp32 product, as a constant
expression, in which an undefined operation does not compile."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_sharded_amd", "csrc")
SOURCE = """
#include "parts.h"
using namespace mps;
// Every pair of parts of which at least the product of the magnitudes 2^-8a and 2^-8b reaches 2^-16, once, and no other.
constexpr bool all_pairs()
{
    int times[3][3] = {};
    for (int i = 0; i < kPairs; ++i) ++times[part_a(i)][part_b(i)];
    for (int a = 0; a < 3; ++a) {
        for (int b = 0; b < 3; ++b) {
            if (times[a][b] != (a + b <= 2 ? 1 : 0)) return false;
        }
    }
    return part_a(kPairs - 1) == 0 && part_b(kPairs - 1) == 0;
}
static_assert(all_pairs(), "");
// Stages are asked for two ahead, also behind the last pair, of which each may be a stage: the address there is one of a part.
constexpr bool behind_the_last()
{
    for (int i = kPairs; i <= kPairs + 2; ++i) {
        if (part_a(i) < 0 || part_a(i) > 2 || part_b(i) < 0 || part_b(i) > 2) return false;
    }
    return true;
}
static_assert(behind_the_last(), "");
int main() { return 0; }
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_pairs_of_parts(tmp_path):
    src = tmp_path / "pairs.cpp"
    src.write_text(SOURCE)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fsyntax-only", "-I", CSRC, str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
