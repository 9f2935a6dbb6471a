"""The launches of the layer with adapters, over all kinds of sizes, without a GPU: tiles, stages and shared memory
within their limits, with the adapters' addends beside the parts of K, and columns of tensor memory covered."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_quantized_moe_router_gb300", "csrc")

PROGRAM = r"""
#include "launch_plan.h"
#include <stdio.h>
using namespace moe;

static long cases = 0, wrong = 0;
template <bool PAIR>
static void few(int T, int N, int K, const LinPlan& p, bool gated) {
    using F = Few<PAIR>;
    ++cases;
    const int parts = few_parts(p.splits, gated, true), smem = F::smem(p.rows_t, p.splits, p.stages, parts);
    const int inner = 1024 + p.stages * F::stage(p.rows_t) + parts * F::kW * F::pitch(F::own(p.rows_t, p.splits)) * 4;
    if (parts < 1 || inner > smem || smem > kCtaSmemMax || !columns_covered(smem, F::columns(p.rows_t)) || p.rows_t > F::kRows ||
        p.rows_t % F::kStep || p.stages < 2 || p.stages > kFewStages || p.splits * F::kCtas > kFewSplits) {
        ++wrong;
        printf("plan of %d %d %d: %d bytes of %d\n", T, N, K, inner, smem);
    }
}
int main() {
    const int Ts[] = {1, 2, 7, 8, 15, 16, 17, 33, 64, 65, 77, 127, 128, 129, 200, 255, 256, 257, 300, 512, 513, 1000, 2048, 4096, 1 << 20, 1 << 30};
    const int Ns[] = {1, 33, 64, 128, 129, 256, 512, 1000, 1536, 2048, 4096, 7168, 20001, 1 << 20};
    const int Ks[] = {8, 64, 72, 256, 776, 1544, 2048, 4096, 7168, 1 << 20};
    for (int T : Ts)
        for (int N : Ns)
            for (int K : Ks)
                for (int gated = 0; gated < 2; ++gated) {
                    const int nk = (K + kLinK - 1) / kLinK;
                    const LinPlan p = plan_linear(T, N, nk, gated, 152, true);
                    if (p.few && p.pair) few<true>(T, N, K, p, gated);
                    if (p.few && !p.pair) few<false>(T, N, K, p, gated);
                    if (!p.few && p.width != 128 && p.width != 192 && p.width != 256) ++wrong;
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
