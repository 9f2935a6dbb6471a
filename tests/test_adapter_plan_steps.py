"""The launches of the low-rank products leave no SMs idle because of a row more, without a GPU: where a group of rows may have more
items than there is room for, whether they are prompts or one row to an adapter, most of the resident CTAs are launched at every length."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_moe_router_gb300", "csrc")

PROGRAM = r"""
#include "launch_plan.h"
#include <initializer_list>
#include <stdio.h>
using namespace moe;

static long cases = 0, wrong = 0;
int main() {
    for (int T = 256; T <= 9000; ++T)
        for (int L : {64, 100, 512, 4096})
            for (int K : {2048, 4096, 7168})
                for (int R : {16, 32, 64})
                    for (int matrices = 1; matrices < 3; ++matrices) {
                        ++cases;
                        const LowPlan p = plan_low_rank(T, K, L, R, matrices);
                        const long ctas = (long)p.groups * p.slots * p.splits;
                        // a batch for each adapter and 32 rows at most, each in passes of 32 ranks
                        const long rows = T < 256 ? T : 256, passes = (R / 16 * matrices + 1) / 2, items = ((L < rows ? L : rows) + rows / 32) * passes;
                        const bool scarce = items * p.groups > 304;
                        if (!scarce || ctas * 3 >= 2 * 304) continue;
                        if (++wrong <= 20) printf("%d rows, K %d, %d adapters of %d, %d: %ld CTAs\n", T, K, L, R, matrices, ctas);
                    }
    printf("%ld cases %ld wrong\n", cases, wrong);
    return 0;
}
"""


def test_no_idle_machine(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    source, program = tmp_path / "steps.cpp", tmp_path / "steps"
    source.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, "-o", str(program), str(source)], check=True)
    out = subprocess.run([str(program)], capture_output=True, text=True, timeout=300, check=True).stdout
    cases, wrong = (int(w) for w in out.split()[-4::2])
    assert wrong == 0, out
    assert cases > 1000
