"""The launches that the clustered tensor-core kernels choose, over all kinds of sizes, without a GPU.

A CTA waits for columns of tensor memory without a limit and holds them while it waits for its cluster.
So CTAs that fit on an SM by shared memory have to fit by columns too (512 of them), whichever kernels and streams they
are of: each takes at least its columns' share of the SM's 228 KB, and one that takes all columns leaves
too little for any other."""
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

static const int kSm = 233472, kCta = 232448, kReserved = 1024, kSmallest = 32 * 456;  // bytes: of an SM, of a CTA at most
static long cases = 0, wrong = 0;
static void check(const char* what, int a, int b, int c, int columns, int smem, int inner) {
    ++cases;
    const bool share = columns == 512 ? smem + kReserved + kSmallest > kSm : (long)(smem + kReserved) * 512 >= (long)columns * kSm;
    if (share && smem + 256 <= kCta && inner <= smem && columns >= 32 && columns <= 512 && !(columns & (columns - 1))) return;
    if (++wrong <= 20) printf("%s %d %d %d: %d columns, %d bytes (needs %d)\n", what, a, b, c, columns, smem, inner);
}
template <bool PAIR>
static void few(int T, int N, int K, const LinPlan& p, bool gated) {
    using F = Few<PAIR>;
    check(gated ? "gated" : "linear", T, N, K, F::columns(p.rows_t), F::smem(p.rows_t, p.splits, p.stages),
          p.stages * F::stage(p.rows_t) + F::rest(p.rows_t, p.splits));
    if (p.rows_t > F::kRows || p.rows_t % F::kStep || p.stages < 2 || p.stages > kFewStages || p.splits * F::kCtas > kFewSplits ||
        F::columns(p.rows_t) < p.rows_t) {
        ++wrong;
        printf("plan of %d %d %d\n", T, N, K);
    }
}
int main() {
    const int Ts[] = {1, 2, 3, 7, 8, 15, 16, 17, 31, 33, 48, 64, 65, 77, 100, 127, 128, 129, 130, 192, 200, 255, 256, 257, 300, 384, 512,
                      513, 700, 1000, 1024, 1500, 2048, 2049, 4096, 5000, 8192, 12000, 16384, 40000, 1 << 20, 1 << 30};
    const int Ns[] = {1, 16, 33, 64, 96, 128, 129, 200, 256, 384, 512, 1000, 1024, 1536, 2048, 2050, 4096, 7168, 8192, 20001, 70000, 1 << 20};
    const int Ks[] = {8, 64, 72, 128, 192, 256, 328, 512, 776, 1024, 1544, 2048, 4096, 7168, 8200, 16384, 1 << 20};
    for (int T : Ts)
        for (int N : Ns)
            for (int K : Ks)
                for (int gated = 0; gated < 2; ++gated) {
                    const LinPlan p = plan_linear(T, N, (K + kLinK - 1) / kLinK, gated, 152);
                    if (p.few && p.pair) few<true>(T, N, K, p, gated);
                    if (p.few && !p.pair) few<false>(T, N, K, p, gated);
                }
    const long linear = cases;
    for (int T : Ts)
        for (int E = 1; E <= 512; ++E)
            for (int H = 32; H <= 8192; H += H < 1024 ? 32 : 512) {
                FusedPlan p{};
                if (!plan_fused(T, E, H, p)) continue;
                const int stage = 128 * 128 + p.n * 128, landing = p.parts * p.own * (p.n + 4) * 4;
                const int inner = 1024 + (p.landing_at ? p.stages * stage : 0) + landing;
                check("route", T, E, H, tmem_columns(p.n), p.smem, inner);
                if (p.stages * stage + 1024 > p.smem || p.scratch_at < p.landing_at + landing || p.n > 256 || p.n * p.blocks < E ||
                    p.own * p.splits < (T < 128 ? T : 128) || p.parts > p.splits || p.parts > p.nk || p.stages > kFusedStagesMax) {
                    ++wrong;
                    printf("plan of route %d %d %d\n", T, E, H);
                }
            }
    printf("%ld linear %ld route %ld wrong\n", linear, cases - linear, wrong);
    return 0;
}
"""


def test_columns_and_shared_memory(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    source, program = tmp_path / "plans.cpp", tmp_path / "plans"
    source.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, "-o", str(program), str(source)], check=True)
    out = subprocess.run([str(program)], capture_output=True, text=True, timeout=300, check=True).stdout
    linear, route, wrong = (int(w) for w in out.split()[-6::2])
    assert wrong == 0, out
    assert linear > 5000 and route > 100000
