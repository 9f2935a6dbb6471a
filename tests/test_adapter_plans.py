"""The launches of the layer with adapters and of its low-rank products, over all kinds of sizes, without a GPU: tiles,
stages and shared memory within their limits, with the adapters' addends beside the parts of K, and columns of tensor memory covered."""
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
template <bool PAIR>
static void few(int T, int N, int K, const LinPlan& p, bool gated) {
    using F = Few<PAIR>;
    ++cases;
    const int own = F::own(p.rows_t, p.splits), parts = few_parts(p.splits, gated, true);
    const int smem = F::smem(p.rows_t, p.splits, p.stages, parts, true);
    const int inner = 1024 + p.stages * F::stage(p.rows_t) + parts * F::kW * F::pitch(own) * 4 + (own + 7) / 8 * 64;
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
    const int Rs[] = {8, 16, 24, 64, 128, 256};
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
    for (int T : Ts)
        for (int L : {1, 2, 5, 8, 33, 64, 100, 128, 1000, 1 << 20})
            for (int K : Ks)
                for (int R : Rs)
                    for (int matrices = 1; matrices < 3; ++matrices) {
                        ++cases;
                        const LowPlan p = plan_low_rank(T, K, L, R, matrices, 152);
                        const int steps = (K + kLowK - 1) / kLowK;
                        const int inner = 1024 + p.stages * p.stage + (p.splits << p.own_log2) * p.width * 4 + 128 * 4;
                        const int reach = 1024 + (p.stages - 1) * p.stage + 128 * 128;
                        const int unit = 1 << p.unit_log2;
                        const bool units = unit >= 16 && p.tile >= 1 && p.tile * unit <= kLowTile && !(p.width & (p.width - 1)) && p.width <= p.tile * unit &&
                                           (1 << p.per_adapter_log2) * unit >= R * matrices && ((1 << p.per_adapter_log2) > p.tile || p.width == (1 << p.per_adapter_log2) * unit);
                        const bool sizes = p.rows % 16 == 0 && p.rows >= 16 && p.rows <= kLowRows && (long)p.rows * p.groups >= T &&
                                           (p.splits << p.own_log2) >= p.rows && p.own_log2 >= 2;
                        const bool ring = p.stages >= 1 && p.stages <= kLowStages && p.splits >= 1 && p.splits <= kLowSplits &&
                                          p.splits <= steps && p.slots >= 1 && p.slots <= 65535 &&
                                          p.loaders >= 1 && p.loaders <= kLowLoaders && p.loaders <= p.stages * p.tile;
                        if (sizes && ring && units && reach <= p.smem && inner <= p.smem && p.smem <= kCtaSmemMax && columns_covered(p.smem, tmem_columns(p.rows))) continue;
                        if (++wrong <= 20) printf("products of %d rows, K %d, %d adapters of %d, %d: %d bytes of %d\n", T, K, L, R, matrices, inner, p.smem);
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
