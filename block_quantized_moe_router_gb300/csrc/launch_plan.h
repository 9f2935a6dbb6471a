// launch_plan.h -- the launches of the clustered tensor-core kernels: tiles, parts of K, ring stages, shared
// memory and columns of tensor memory per CTA (internal).  Plain C++ without CUDA headers, so that the rule on
// columns is tested over all sizes on the CPU (tests/test_launch_plans.py).
#pragma once
#include <stdint.h>

namespace moe {

// ---- tensor memory and shared memory ----------------------------------------------------------
// A CTA waits for its columns of tensor memory without a limit (tcgen05.alloc has none), and a CTA of a cluster
// holds them while it waits for the cluster's other CTAs.  Were two SMs to hold more CTAs than they have
// columns for, clusters of several streams could each hold columns on one and wait for the other's on the
// other, for ever.  So a CTA that takes a share of the columns takes at least that share of the SM's shared memory: CTAs
// that fit by shared memory fit by columns, whatever their kernels and registers.
// CTAs without a cluster (prefill_tc.cu) hold theirs only while they run on, and wait for nobody then.
constexpr int kSmSmem = 228 * 1024;       // shared memory of an SM
constexpr int kCtaSmemMax = 226 * 1024;   // dynamic shared memory of a CTA here
constexpr int kSmemReserved = 1024;       // taken per CTA besides
constexpr int kTmemColumns = 512;
constexpr int kTmemLeast = 32;            // columns are allocated in powers of two from here on
constexpr int kColumnSmem = kSmSmem / kTmemColumns;
constexpr int tmem_columns(int n) {
    int c = kTmemLeast;
    while (c < n) c *= 2;
    return c;
}
// The least dynamic shared memory of a CTA with so many columns.
constexpr int smem_for_columns(int columns) {
    const int least = columns * kColumnSmem - kSmemReserved;
    return least < kCtaSmemMax ? least : kCtaSmemMax;
}
// Whether the rule holds; with all columns, that no CTA with any fits beside.
constexpr bool columns_covered(int smem, int columns) {
    return columns == kTmemColumns ? smem + kSmemReserved + kTmemLeast * kColumnSmem > kSmSmem
                                   : smem + kSmemReserved >= columns * kColumnSmem;
}

// ---- moe_linear ---------------------------------------------------------------------------------
constexpr int kLinK = 64;        // K elements per stage (128 bytes per row)
constexpr int kFewSplits = 8;    // parts of K at most; CTAs of a cluster too (the portable cluster size)
constexpr int kFewStages = 8;
template <bool PAIR>
struct Few {
    static constexpr int kRows = PAIR ? 256 : 128;   // rows of x per tile at most
    static constexpr int kStep = PAIR ? 32 : 16;     // a tile's rows of x are a multiple of it
    static constexpr int kW = PAIR ? 64 : 128;       // weight rows of a CTA
    static constexpr int kA = kW * 128;              // bytes of them per stage
    static constexpr int kCtas = PAIR ? 2 : 1;       // per part of K
    static constexpr int own(int rows, int splits) { return ((rows + splits - 1) / splits + 3) / 4 * 4; }
    static constexpr int pitch(int own) { return own | 4; }  // own is a multiple of 4
    static constexpr int stage(int rows) { return kA + rows / kCtas * 128; }
    // A pair takes all of tensor memory, so that its CTAs hold the same columns.
    static constexpr int columns(int rows) { return PAIR ? kTmemColumns : tmem_columns(rows); }
    static constexpr int rest(int rows, int splits) {  // beside the stages
        return splits * kW * pitch(own(rows, splits)) * 4 + 1024;
    }
    static constexpr int smem(int rows, int splits, int stages) {
        const int need = stages * stage(rows) + rest(rows, splits);
        const int least = smem_for_columns(columns(rows));
        return need > least ? need : least;
    }
};

// Tiles of the many-row kernel: 256 rows by `features`.
constexpr int64_t many_tiles(int T, int N, int features) {
    return ((int64_t)T + 255) / 256 * ((N + features - 1) / features);
}

// Which kernel, and its tiles, by estimated time in microseconds.  The constants are fitted to all the choices
// at 168 sizes (1 to 4096 rows, N 88 to 7168, K 512 to 7168); the choices that nearby constants make are 1 %
// faster in the mean at best, 20 % at single sizes.
//   many rows: tiles go out in waves of one per CTA pair; 64 elements of K cost 0.38 / 0.31 / 0.25 us
//     at 256 / 192 / 128 columns (the loads of x do not shrink with the columns), 0.95 us a tile
//     besides, and 3 us once.  512 x 7168 x 2048: 18.2 us at 192 columns (one wave), 19.8 at 256.
//   few rows: 64 elements cost a CTA 0.2 us, in pairs 0.22, or what its SM's share of the L2 rate (106 GB/s)
//     allows; every row of x costs its exchange and sums, least where a part of K has a tile alone; 1.6 us
//     a wave and 0.6 us once besides.  128 rows of the gated 2 x 2048 x 7168: 16.2 us in two parts by pairs,
//     19.3 in four by single CTAs, 31.2 in the other kernel; 256 rows of 7168 x 2048: 15.4, 17.4 and 14.7.
struct LinPlan {
    bool few, pair;
    int width;                   // many: columns per tile
    int splits, stages, rows_t;  // few: parts of K, ring stages, rows of x per tile
};

// Of 152 SMs, how many places for one CTA each clusters can use: 36 clusters of 4 and 15 of 8 are resident at
// one CTA per SM, 36 of 8 at two.
constexpr int few_usable(int cluster, int fit) { return cluster < 4 ? 152 : cluster == 8 && fit == 1 ? 120 : 144; }

// The few-row choices with the rows of x in `tiles_t` tiles.
template <bool PAIR>
void plan_few_tiles(int T, int N, int nk, bool gated, int sms, int tiles_t, float& best_us, LinPlan& best) {
    using F = Few<PAIR>;
    const int rows = ((T + tiles_t - 1) / tiles_t + F::kStep - 1) / F::kStep * F::kStep;
    const int per_tile = F::kW * F::kCtas / (gated ? 2 : 1);
    const int64_t tiles = (int64_t)((T + rows - 1) / rows) * ((N + per_tile - 1) / per_tile) * F::kCtas;
    const float stage_kb = (float)F::stage(rows) / 1024.f;
    for (int splits = 1; splits * F::kCtas <= kFewSplits && splits <= nk; splits *= 2) {
        const int kbs = (nk + splits - 1) / splits;
        // Pairs and CTAs alone on their SMs take more stages, so that latency from HBM does not hold the loads
        // back (64 rows of 7168 x 2048: 12.1 us with 4, 11.4 with 6; with 8 what follows starts later).
        const bool alone = PAIR || tiles * splits <= (int64_t)sms * few_usable(splits, 1) / 152;
        int stages = alone ? (kCtaSmemMax - F::rest(rows, splits)) / F::stage(rows) : 4;
        const int most = PAIR ? kFewStages : alone ? 6 : 4;
        stages = stages < most ? stages : most;
        stages = kbs < stages ? (kbs < 2 ? 2 : kbs) : stages;
        const int smem = F::smem(rows, splits, stages);
        if (stages < 2 || smem > kCtaSmemMax) continue;
        const int fit = kSmSmem / (smem + kSmemReserved + 256);  // CTAs an SM holds
        const int64_t places = (int64_t)sms * fit * few_usable(splits * F::kCtas, fit) / 152;
        const int64_t ctas = tiles * splits, waves = (ctas + places - 1) / places;
        const int64_t on_sm = waves > 1 ? fit : (ctas + sms - 1) / sms;
        const float per_k_lat = PAIR ? 0.22f : 0.2f, per_k_bw = (float)on_sm * stage_kb / 106.f;
        const float per_row = splits == 1 && !gated ? (PAIR ? 0.012f : 0.037f) : (PAIR ? 0.0175f : 0.051f);
        const float us = (float)waves * ((float)kbs * (per_k_bw > per_k_lat ? per_k_bw : per_k_lat) +
                                         per_row * (float)rows + 1.6f) + (PAIR ? 0.65f : 0.6f);
        if (us < best_us) {
            best_us = us;
            best = LinPlan{true, PAIR, 0, splits, stages, rows};
        }
    }
}
// As few tiles of x as its rows need, or up to eight times as many where a narrow matrix leaves SMs idle
// (256 x 2048 x 2048: 12.9 us with one, 10.0 with two; 128 x 256 x 7168: 9.5 with one, 5.9 with four).
template <bool PAIR>
void plan_few(int T, int N, int nk, bool gated, int sms, float& best_us, LinPlan& best) {
    using F = Few<PAIR>;
    const int least = (T + F::kRows - 1) / F::kRows;
    for (int m = 1; m <= 8 && (m == 1 || least * m * F::kStep < T + F::kStep) && least * m <= 65535; m *= 2)
        plan_few_tiles<PAIR>(T, N, nk, gated, sms, least * m, best_us, best);
}

inline LinPlan plan_linear(int T, int N, int nk, bool gated, int sms) {
    LinPlan best{};
    float best_us = 1e30f;
    const float per_k[3] = {0.38f, 0.31f, 0.25f};
    for (int i = 0; i < 3; ++i) {
        const int width = 256 - 64 * i;
        const int64_t tiles = many_tiles(T, N, gated ? width / 2 : width);
        const int64_t waves = (tiles + sms / 2 - 1) / (sms / 2);
        const float us = (float)waves * ((float)nk * per_k[i] + 0.95f) + 3.f;
        if (us < best_us) {
            best_us = us;
            best = LinPlan{false, false, width, 0, 0, 0};
        }
    }
    plan_few<false>(T, N, nk, gated, sms, best_us, best);
    plan_few<true>(T, N, nk, gated, sms, best_us, best);
    return best;
}

// ---- moe_route_grouped --------------------------------------------------------------------------
// Shared memory of one routing warp.
template <int EPL>
struct alignas(16) RouteScratch {
    // Ranking values, size + 1 places per group: value e stands at e + e / size, also for e from E to
    // 32 EPL - 1.  With at most 64 groups and E > 16 EPL the groups are of at least 2, 3 and 5 experts at EPL
    // 4, 8 and 16, which puts the last place at 190, 340 and 613 (EPL 1 and 2: groups of one, 62 and 126).
    float rank[32 * EPL + (EPL == 1 ? 32 : EPL <= 4 ? 64 : EPL == 8 ? 96 : 112)];
    float val[32 * EPL];  // scores (logits where no score was needed, or for fp64)
    float group[68];
    int kept[64];
};

constexpr int route_scratch_bytes(int E) {
    return (int)(E <= 32 ? sizeof(RouteScratch<1>) : E <= 64 ? sizeof(RouteScratch<2>) : E <= 128 ? sizeof(RouteScratch<4>)
                                                                                         : sizeof(RouteScratch<8>));
}

constexpr int kFusedThreads = 512;
constexpr int kFusedK = 64;
constexpr int kFusedA = 128 * 128;
constexpr int kFusedStagesMax = 8;

struct FusedPlan {
    int blocks, n, nk;      // blocks of experts; n: experts of one rounded up to 16, the MMA's columns; stages of K
    int splits, parts;      // CTAs of a cluster, and those of them that have a part of K
    int own, stages;        // tokens per CTA of a tile; ring stages
    int box_x;              // token rows a TMA box brings
    int landing_at;         // byte offsets: of the landing area (0: over the ring)
    int scratch_at;         // and of the warps' scratch
    int smem;
};

// false where the router's own kernels are faster.
inline bool plan_fused(int T, int E, int H, FusedPlan& p) {
    p.blocks = (E + 255) / 256;
    // Two launches save none, and a small product is done sooner without clusters: 1 x 512 x 2048 7.5 us
    // against 8.9 (1 x 384 x 7168 10.7 against 9.4), 161 x 466 x 352 9.9 against 15.6 (2702 tokens 28.8 against
    // 20.9; 16 x 512 x 2048 33.3 against 9.5).
    if (p.blocks > 1 && (T == 1 ? H <= 4096 : T <= 1024 && H <= 512)) return false;
    p.nk = (H + kFusedK - 1) / kFusedK;
    p.n = ((E + p.blocks - 1) / p.blocks + 15) / 16 * 16;
    // as many CTAs per tile as keep every cluster resident at one CTA per SM (152 SMs hold 7, 15,
    // 36 and 76 clusters of 16, 8, 4 and 2), but beyond one per stage only to share many tokens
    const int64_t tiles = ((int64_t)T + 127) / 128 * p.blocks;
    const int rows = T < 128 ? T : 128;
    p.splits = tiles <= 7 ? 16 : tiles <= 15 ? 8 : tiles <= 36 ? 4 : tiles <= 76 ? 2 : 1;
    while (p.splits > p.nk && rows <= p.splits / 2 * (kFusedThreads / 32)) p.splits /= 2;
    p.parts = p.splits < p.nk ? p.splits : p.nk;
    p.own = (rows + p.splits - 1) / p.splits;
    p.box_x = (rows + 7) / 8 * 8;
    // ring | landing | scratch, or the last two over the ring where they do not fit beside it
    const int stage = kFusedA + p.n * 128;
    const int landing = p.parts * p.own * (p.n + 4) * 4;
    const int warps = p.own < kFusedThreads / 32 ? p.own : kFusedThreads / 32;
    const int scratch = p.blocks == 1 ? route_scratch_bytes(E) * warps : 0;
    const int steps = (p.nk + p.parts - 1) / p.parts;
    const int landing16 = (landing + 15) / 16 * 16;
    p.stages = (kCtaSmemMax - 1024 - landing16 - scratch) / stage;
    const bool beside = p.stages >= 3 || p.stages >= steps;
    if (!beside) p.stages = (kCtaSmemMax - 1024) / stage;
    p.stages = p.stages < steps ? p.stages : steps;
    p.stages = p.stages < 1 ? 1 : p.stages < kFusedStagesMax ? p.stages : kFusedStagesMax;
    p.landing_at = beside ? p.stages * stage : 0;
    p.scratch_at = p.landing_at + landing16;
    p.smem = p.scratch_at + scratch;
    if (p.stages * stage > p.smem) p.smem = p.stages * stage;
    p.smem += 1024;
    const int least = smem_for_columns(tmem_columns(p.n));
    if (p.smem < least) p.smem = least;
    return p.smem <= kCtaSmemMax;
}

}  // namespace moe
