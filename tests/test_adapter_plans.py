"""The launches of the low-rank products of a layer with adapters, over all kinds of sizes, without a GPU: groups cover the rows, and
slots, parts of K and landing areas stay within their limits."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_quantized_moe_router_gb300", "csrc")

PROGRAM = r"""
#include "launch_plan.h"
#include <initializer_list>
#include <stdio.h>
using namespace moe;

static long cases = 0, wrong = 0;
int main() {
    for (int T : {1, 2, 7, 8, 31, 32, 33, 77, 128, 255, 256, 257, 300, 512, 1000, 2107, 4096, 65536, 1 << 24, 1 << 30})
        for (int L : {1, 2, 5, 8, 33, 96, 100, 128, 1000, 1 << 20})
            for (int K : {8, 64, 72, 256, 512, 776, 1544, 2048, 2632, 4096, 7168, 1 << 20})
                for (int R : {8, 16, 24, 48, 64, 128, 256})
                    for (int matrices = 1; matrices < 3; ++matrices) {
                        ++cases;
                        const LowPlan p = plan_low_rank(T, K, L, R, matrices);
                        const int steps = (K + 31) / 32;
                        const bool sizes = (long)p.groups * kLowGroup >= T && (long)(p.groups - 1) * kLowGroup < T && p.slots >= 1 &&
                                           (long)p.slots * p.splits <= 65536 && p.landing_rows >= 1 && p.landing_rows <= kLowBatch && p.landing_rows <= T;
                        const bool parts = p.splits >= 1 && p.splits <= kLowSplits && !(p.splits & (p.splits - 1)) && p.splits <= steps &&
                                           p.smem <= kLowLandingMax && (p.splits == 1 || p.smem == p.splits * p.landing_rows * kLowRanks * 4);
                        if (sizes && parts) continue;
                        if (++wrong <= 20) printf("products of %d rows, K %d, %d adapters of %d, %d: %d slots, %d parts, %d bytes\n", T, K, L, R, matrices, p.slots, p.splits, p.smem);
                    }
    printf("%ld cases %ld wrong\n", cases, wrong);
    return 0;
}
"""


def test_plans(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    source, program = tmp_path / "plans.cpp", tmp_path / "plans"
    source.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, "-o", str(program), str(source)], check=True)
    out = subprocess.run([str(program)], capture_output=True, text=True, timeout=300, check=True).stdout
    cases, wrong = (int(w) for w in out.split()[-4::2])
    assert wrong == 0, out
    assert cases > 1000
