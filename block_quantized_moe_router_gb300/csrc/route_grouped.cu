// route_grouped.cu -- top-K routing limited to expert groups.
//
// The E experts form n_group groups of E / n_group consecutive ids.  With scores s = softmax,
// sigmoid or sqrt(softplus) of the logits and v = s + bias (the bias selects only):
//   G_g  = sum of the group_top (1 or 2) largest v of group g
//   keep = the topk_group groups with the largest G            (ties: lower group)
//   ids  = the top_k largest v among the experts of the kept groups (ties: lower expert)
//   w_j  = s_j / sum of the picked s * scaling   (renormalised)   or   s_j * scaling
//
// The order is that of the exact values.  fp32 scores carry an error of some 2^-22 of their
// size, so two scores closer than a bound on that error could be picked the wrong way round;
// where a comparison that decides the result falls inside the bound, the values concerned are
// computed again in fp64.  Without a bias every score grows with its logit, and experts are ranked by
// the logits themselves, which needs no bound.
//
// One warp routes one token (lane l holds experts l, l + 32, ...).  Only the kept groups' experts
// go into the K rounds, dealt anew over the lanes, so a round looks at topk_group / n_group of the
// values.
#include <cudaTypedefs.h>

#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch_plan.h"
#include "tc_ptx.cuh"
#include "topk.cuh"

namespace moe {

namespace {

struct GroupRule {
    int E, k, scoring, renorm, n_group, topk_group, group_top, by_logit;
    int size;       // experts per group
    int size_inv;   // ceil(2^20 / size): (r * size_inv) >> 20 == r / size for r < 512
    int group_lanes, group_shift;  // lanes that share a group, the largest power of two <= 32 / n_group
    float scaling;
};

template <int V>
struct Int {
    static constexpr int value = V;
};

__device__ __forceinline__ bool is_softmax(int scoring) {
    return scoring == MOE_SCORE_SOFTMAX || scoring == MOE_SCORE_SOFTMAX_BIAS;
}

// Score of a finite logit.  fp32: expf and __fdividef are within 2 units in the last place each, but the quotient is 0 where
// its divisor passes 2^126, so a sigmoid below 2^-126 (a logit below -87.3) reads as 0; a softmax score below that
// may be subnormal.  log(1 + e^l) is e^l to within e^l / 2 of itself, so far below 0 sqrt(softplus) is e^(l/2): e^l would
// be subnormal, and its root off by more than fp32 holds, from l = -87 on.
__device__ __forceinline__ float score32(int scoring, float l, float lmax, float inv_z) {
    if (is_softmax(scoring)) return expf(l - lmax) * inv_z;
    if (scoring == MOE_SCORE_SQRTSOFTPLUS) return l < -20.f ? expf(0.5f * l) : sqrtf(l > 30.f ? l : log1pf(expf(l)));
    return __fdividef(1.f, 1.f + expf(-l));
}
__device__ __forceinline__ double score64(int scoring, double l, double lmax, double inv_z) {
    if (is_softmax(scoring)) return exp(l - lmax) * inv_z;
    if (scoring == MOE_SCORE_SQRTSOFTPLUS) return l < -40. ? exp(0.5 * l) : sqrt(l > 40. ? l : log1p(exp(l)));
    return 1. / (1. + exp(-l));
}

__device__ __forceinline__ float from_orderable(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
// fp64 -> uint64 with the same order as the values (0 is below every value)
__device__ __forceinline__ unsigned long long orderable64(double v) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.);  // -0 and +0 are equal
    return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ double from_orderable64(unsigned long long u) {
    return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}

// 1 / softmax denominator over the finite logits in sc->val, in fp64.
template <int EPL>
__device__ __forceinline__ double inv_z64(const GroupRule& P, float lmax, const RouteScratch<EPL>* sc, int lane) {
    if (!is_softmax(P.scoring)) return 1.;
    double z = 0.;
    for (int e = lane; e < P.E; e += 32)
        if (sc->val[e] != -INFINITY) z += exp((double)sc->val[e] - (double)lmax);
#pragma unroll
    for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    return 1. / z;
}

// The ranking value of expert e in fp64 as an ordered key, from the logits in sc->val.
template <int EPL>
__device__ __forceinline__ unsigned long long key_of(const GroupRule& P, const float* bias, int e, float lmax,
                                                     double inv_z, const RouteScratch<EPL>* sc) {
    const float l = sc->val[e], b = bias ? bias[e] : 0.f;
    if (l == -INFINITY || !isfinite(b)) return orderable64(-INFINITY);
    if (P.by_logit) return orderable64(l);
    return orderable64(score64(P.scoring, l, lmax, inv_z) + (double)b);
}

// Which of the groups in `close` are kept, `room` of them, by their scores in fp64, from the logits in
// sc->val.
template <int EPL>
__device__ __noinline__ unsigned long long kept_fp64(const GroupRule& P, const float* bias, float lmax,
                                                     unsigned long long close, int room,
                                                     const RouteScratch<EPL>* sc, int lane) {
    const double inv_z = inv_z64<EPL>(P, lmax, sc, lane);
    unsigned long long mine[2] = {0, 0}, kept = 0;
    for (unsigned long long left = close; left; left &= left - 1) {
        const int g = __ffsll((long long)left) - 1;
        unsigned long long m1 = 0, m2 = 0;
        for (int i = lane; i < P.size; i += 32) {
            const int e = g * P.size + i;
            const float l = sc->val[e];
            const unsigned long long x =
                P.by_logit && P.group_top == 2 && l != -INFINITY
                    ? orderable64(score64(P.scoring, l, lmax, inv_z))
                    : key_of<EPL>(P, bias, e, lmax, inv_z, sc);
            m2 = max(m2, min(m1, x));
            m1 = max(m1, x);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const unsigned long long b1 = __shfl_xor_sync(0xffffffffu, m1, o);
            const unsigned long long b2 = __shfl_xor_sync(0xffffffffu, m2, o);
            m2 = max(min(m1, b1), m1 > b1 ? m2 : b2);
            m1 = max(m1, b1);
        }
        const unsigned long long key =
            P.group_top == 2 ? orderable64(from_orderable64(m1) + from_orderable64(m2)) : m1;
        if (lane == (g & 31)) mine[g >> 5] = key;
    }
    for (unsigned long long left = close; left; left &= left - 1) {
        const int g = __ffsll((long long)left) - 1;
        const unsigned long long x = __shfl_sync(0xffffffffu, g < 32 ? mine[0] : mine[1], g & 31);
        const bool a0 = ((close >> lane) & 1) && (mine[0] > x || (mine[0] == x && lane < g));
        const bool a1 = ((close >> (lane + 32)) & 1) && (mine[1] > x || (mine[1] == x && lane + 32 < g));
        const int rank = __popc(__ballot_sync(0xffffffffu, a0)) + __popc(__ballot_sync(0xffffffffu, a1));
        if (rank < room) kept |= 1ull << g;
    }
    return kept;
}

// The K rounds in fp64 (more candidates are too close together than a warp's lanes rank), over the
// kept groups, from the logits in sc->val.  On return lane j < k holds pick j.
template <int EPL>
__device__ __noinline__ int pick_fp64(const GroupRule& P, const float* bias, float lmax, RouteScratch<EPL>* sc,
                                      int lane) {
    const double inv_z = inv_z64<EPL>(P, lmax, sc, lane);
    const bool grouped = P.topk_group < P.n_group;
    const int count = grouped ? P.topk_group * P.size : P.E;
    unsigned long long key[EPL];
    int ee[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int r = lane + 32 * j;
        key[j] = 0;
        ee[j] = 0x7fffffff;
        if (r >= count) continue;
        const int q = (r * P.size_inv) >> 20;
        ee[j] = grouped ? sc->kept[q] * P.size + r - q * P.size : r;
        key[j] = key_of<EPL>(P, bias, ee[j], lmax, inv_z, sc);
    }
    int my_e = 0;
    for (int r = 0; r < P.k; ++r) {
        unsigned long long m = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) m = max(m, key[j]);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(m >> 32));
        const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(m >> 32) == hi ? (uint32_t)m : 0u);
        const unsigned long long top = ((unsigned long long)hi << 32) | lo;
        uint32_t e = 0x7fffffffu;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (key[j] == top) e = min(e, (uint32_t)ee[j]);
        e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (ee[j] == (int)e) key[j] = 0;
        if (lane == r) my_e = (int)e;
    }
    return my_e;
}

// The score in fp64 of the pick with logit l (lanes below k) over the sum of them all; 0 where that sum is 0 too.  The
// softmax's denominator drops out.
__device__ __noinline__ float weight_fp64(int scoring, float l, float lmax, bool pick) {
    const double s = pick && fabsf(l) < INFINITY ? score64(scoring, l, lmax, 1.) : 0.;
    double den = s;
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    return den > 0. ? (float)(s / den) : 0.f;
}

// The K rounds over `count` candidates, N per lane: candidate r is expert r, or the r-th of the kept
// groups.  Returns the pick of lane j < k, or sets `full` where all candidates are needed in fp64.
template <int EPL, int N>
__device__ __forceinline__ int pick_rounds(const GroupRule& P, const float* bias, RouteScratch<EPL>* sc, int lane,
                                           bool grouped, float tol_rel, float tol_abs, float lmax,
                                           const float (&lg)[EPL], bool& full, bool& val_is_logit) {
    const float* rank_val = sc->rank;
    const int count = grouped ? P.topk_group * P.size : P.E;
    uint32_t key[N];
    int ee[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int r = lane + 32 * j;
        key[j] = 0;  // below every value
        ee[j] = 0x7fffffff;
        if (r < count) {
            const int q = (r * P.size_inv) >> 20;
            const int g = grouped ? sc->kept[q] : q;
            ee[j] = g * P.size + r - q * P.size;
            key[j] = orderable(rank_val[ee[j] + g]);  // a group takes size + 1 places: no bank conflicts
        }
    }
    int r = 0, want = P.k, my_e = 0;
    uint32_t my_key = 0;
    for (bool again = false;; again = true) {
        for (; r < want; ++r) {
            uint32_t m = key[0];
#pragma unroll
            for (int j = 1; j < N; ++j) m = max(m, key[j]);
            const uint32_t top = __reduce_max_sync(0xffffffffu, m);
            uint32_t e = 0x7fffffffu;  // the lowest expert that reaches the top
#pragma unroll
            for (int j = N - 1; j >= 0; --j) e = key[j] == top ? (uint32_t)ee[j] : e;
            e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
            for (int j = 0; j < N; ++j) key[j] = ee[j] == (int)e ? 0u : key[j];
            my_e = lane == r ? (int)e : my_e;
            my_key = lane == r ? top : my_key;
        }
        if (P.by_logit) return my_e;
        // neighbours too close, or one left behind too close to the last pick that counts?
        const float v = from_orderable(my_key);
        const float tol = 2.f * (tol_rel * fabsf(v) + tol_abs);
        const float before = __shfl_up_sync(0xffffffffu, v, 1);
        const bool near = lane > 0 && lane < P.k && v > -INFINITY && before - v <= tol;
        const float bar = __shfl_sync(0xffffffffu, v - tol, P.k - 1);
        bool left = false;
#pragma unroll
        for (int j = 0; j < N; ++j) left = left || (bar > -INFINITY && key[j] >= orderable(bar));
        left = __any_sync(0xffffffffu, left);
        if (!again) {
            if (!left && !__any_sync(0xffffffffu, near)) return my_e;
            // a few candidates more, and the order among all these in fp64
            val_is_logit = true;
            want = min(min(P.k + 4, 32), count);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (lane + 32 * j < P.E) sc->val[lane + 32 * j] = lg[j];
            __syncwarp();
        } else {
            if (left) {  // more than those are that close
                full = true;
                return 0;
            }
            const double inv_z = inv_z64<EPL>(P, lmax, sc, lane);
            const unsigned long long mine = lane < want ? key_of<EPL>(P, bias, my_e, lmax, inv_z, sc) : 0;
            int rank = 0;
            for (int i = 0; i < want; ++i) {
                const unsigned long long o = __shfl_sync(0xffffffffu, mine, i);
                const int oe = __shfl_sync(0xffffffffu, my_e, i);
                rank += o > mine || (o == mine && oe < my_e) ? 1 : 0;
            }
            __syncwarp();
            if (lane < want) sc->kept[rank] = my_e;
            __syncwarp();
            return lane < P.k ? sc->kept[lane] : 0;
        }
    }
}

// One warp routes one token: raw[j] and bv[j] are the logit and the bias of expert lane + 32 j (anything
// beyond E), `logits` its row in memory, read again where weights underflow (raw kept in registers until then: 26.1 -> 28.2
// us for 8192 rows of 512, 26.3 so).  The branches on the kind of scores stand outside the loops over j: a warp on its own
// spends some twenty cycles on each.
template <int EPL>
__device__ __forceinline__ void route_token(const GroupRule& P, const float (&raw)[EPL], const float (&bv)[EPL],
                                            const float* logits, const float* bias, RouteScratch<EPL>* sc, int lane,
                                            int32_t* ids, float* wout, int32_t* status) {
    const bool softmax = is_softmax(P.scoring), grouped = P.topk_group < P.n_group;
    float lg[EPL], lmax = -INFINITY;
    bool nonfinite = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const bool in = lane + 32 * j < P.E, fin = fabsf(raw[j]) < INFINITY;
        nonfinite |= in & !fin;
        lg[j] = in & fin ? raw[j] : -INFINITY;
        lmax = fmaxf(lmax, lg[j]);
    }
    if (__any_sync(0xffffffffu, nonfinite) && lane == 0) status_or(status, MOE_DEV_NONFINITE);

    const bool need_score = !P.by_logit || (grouped && P.group_top == 2);
    const bool score_groups = grouped && P.by_logit && P.group_top == 2;  // groups add scores, experts rank by logit
    float s[EPL], inv_z = 1.f, smax = 0.f;
    if (need_score || softmax) lmax = from_orderable(__reduce_max_sync(0xffffffffu, orderable(lmax)));
    const float top_logit = lmax == -INFINITY ? 0.f : lmax;
    if (softmax && (need_score || !P.renorm)) {
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            s[j] = expf(lg[j] - top_logit);  // 0 for -inf
            z += s[j];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        inv_z = z > 0.f ? __fdividef(1.f, z) : 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] *= inv_z;
        smax = inv_z;
    } else if (need_score && P.scoring == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] = __fdividef(1.f, 1.f + expf(-lg[j]));
        smax = __fdividef(1.f, 1.f + expf(-top_logit));
    } else if (need_score) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] = score32(P.scoring, lg[j], lmax, inv_z);
        smax = score32(P.scoring, top_logit, lmax, inv_z);
    }
    // places beyond E are written too: the arrays have room, and nothing reads them
    float* rank_val = sc->rank;
    float bmax = 0.f;
    if (P.by_logit) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 32 * j;
            const float v = lg[j] + 0.f;  // -0 and +0 are equal
            rank_val[e + ((e * P.size_inv) >> 20)] = score_groups && lg[j] != -INFINITY ? s[j] : v;
            sc->val[e] = need_score ? s[j] : lg[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 32 * j;
            const bool ok = fabsf(bv[j]) < INFINITY;
            rank_val[e + ((e * P.size_inv) >> 20)] = ok & (lg[j] != -INFINITY) ? s[j] + bv[j] : -INFINITY;
            sc->val[e] = s[j];
            bmax = fmaxf(bmax, ok ? fabsf(bv[j]) : 0.f);
        }
    }
    // Error bounds of a ranking value v: exp, sums and the reciprocal are within 2^-21 of the largest
    // score and of |v|, and what underflow takes is below 2^-126; an error of the softmax denominator (2^-19.7 for 512
    // logits) scales all scores alike, so between close values it counts only with what their scores differ by: no more than the
    // largest score, nor than their biases differ (without the former a single bias of -1e9 sent every token to fp64,
    // 32768 rows of 128 in 828 us).
    const float tol_rel = 0x1p-21f;
    float tol_abs = 2.f * tol_rel * smax + 0x1p-125f;
    if (softmax && !P.by_logit)
        tol_abs += 0x1p-19f * fminf(smax, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(bmax))));

    bool full = false, val_is_logit = !need_score;  // full: see pick_rounds; val_is_logit: sc->val holds logits
    __syncwarp();
    if (grouped) {
        // 32 / n_group lanes (a power of two) share a group; above 32 groups a lane has two
        const int per = P.group_lanes;
        const bool two = P.n_group > 32;
        float gs[2] = {-INFINITY, -INFINITY}, tol[2] = {};
        const auto scan = [&](int q) {
            const int g = (lane >> P.group_shift) + 32 * q;
            const bool in = g < P.n_group;
            float m1 = -INFINITY, m2 = -INFINITY;
            const float* src = rank_val + (in ? g : 0) * (P.size + 1);
#pragma unroll 4
            for (int i = lane & (per - 1); i < P.size; i += per) {
                const float x = src[i];
                m2 = fmaxf(m2, fminf(m1, x));
                m1 = fmaxf(m1, x);
            }
            for (int o = per >> 1; o; o >>= 1) {
                const float b1 = __shfl_xor_sync(0xffffffffu, m1, o);
                const float b2 = __shfl_xor_sync(0xffffffffu, m2, o);
                m2 = fmaxf(fminf(m1, b1), m1 > b1 ? m2 : b2);
                m1 = fmaxf(m1, b1);
            }
            // half of the sum, which does not pass the largest number (-infinity is for what is not finite)
            gs[q] = P.group_top == 2 ? 0.5f * m1 + 0.5f * m2 : m1;
            tol[q] = tol_rel * (P.group_top == 2 ? 0.5f * fabsf(m1) + 0.5f * fabsf(m2) : fabsf(m1)) + tol_abs;
            if (in) sc->group[g] = gs[q];  // the lanes of a group write the same
        };
        scan(0);
        if (two) scan(1);
        if (lane < 3) sc->group[P.n_group + lane] = NAN;  // counts for nothing
        __syncwarp();
        unsigned long long kept = 0;
        bool in[2] = {false, false}, keep[2] = {false, false};
        float lo = INFINITY, hi = -INFINITY;
        const auto place = [&](int q) {
            const int g = (lane >> P.group_shift) + 32 * q;
            int rank = 0;  // the lanes of a group share the comparisons
            for (int i = 4 * (lane & (per - 1)); i < P.n_group; i += 4 * per) {
                const float4 o = *reinterpret_cast<const float4*>(sc->group + i);
                rank += (int)((o.x > gs[q]) | ((o.x == gs[q]) & (i < g)));
                rank += (int)((o.y > gs[q]) | ((o.y == gs[q]) & (i + 1 < g)));
                rank += (int)((o.z > gs[q]) | ((o.z == gs[q]) & (i + 2 < g)));
                rank += (int)((o.w > gs[q]) | ((o.w == gs[q]) & (i + 3 < g)));
            }
            for (int o = per >> 1; o; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
            in[q] = ((lane & (per - 1)) == 0) & (g < P.n_group);
            keep[q] = in[q] & (rank < P.topk_group);
            lo = keep[q] ? fminf(lo, gs[q] - tol[q]) : lo;
            hi = in[q] & !keep[q] ? fmaxf(hi, gs[q] + tol[q]) : hi;
        };
        place(0);
        if (two) place(1);
        if (need_score) {
            lo = from_orderable(__reduce_min_sync(0xffffffffu, orderable(lo)));
            hi = from_orderable(__reduce_max_sync(0xffffffffu, orderable(hi)));
        }
        if (need_score && hi > -INFINITY && lo > -INFINITY && hi >= lo) {
            // the border runs between groups too close to tell: those again in fp64
            unsigned long long sure = 0, close = 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const bool c = in[q] && (keep[q] ? gs[q] - tol[q] <= hi : gs[q] + tol[q] >= lo);
                const int g = (lane >> P.group_shift) + 32 * q;
                const unsigned long long bit = 1ull << (g & 63);
                close |= c ? bit : 0ull;
                sure |= keep[q] && !c ? bit : 0ull;
            }
            close = __reduce_or_sync(0xffffffffu, (unsigned)close) |
                    (unsigned long long)__reduce_or_sync(0xffffffffu, (unsigned)(close >> 32)) << 32;
            sure = __reduce_or_sync(0xffffffffu, (unsigned)sure) |
                   (unsigned long long)__reduce_or_sync(0xffffffffu, (unsigned)(sure >> 32)) << 32;
            val_is_logit = true;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (lane + 32 * j < P.E) sc->val[lane + 32 * j] = lg[j];
            __syncwarp();
            kept = sure | kept_fp64<EPL>(P, bias, lmax, close, P.topk_group - __popcll(sure), sc, lane);
            if (lane < P.n_group && ((kept >> lane) & 1)) sc->kept[__popcll(kept & ((1ull << lane) - 1))] = lane;
            if (lane + 32 < P.n_group && ((kept >> (lane + 32)) & 1))
                sc->kept[__popcll(kept & ((1ull << (lane + 32)) - 1))] = lane + 32;
        } else {
            const unsigned b0 = __ballot_sync(0xffffffffu, keep[0]), below = (1u << lane) - 1u;
            if (keep[0]) sc->kept[__popc(b0 & below)] = lane >> P.group_shift;
            if (two) {
                const unsigned b1 = __ballot_sync(0xffffffffu, keep[1]);
                if (keep[1]) sc->kept[__popc(b0) + __popc(b1 & below)] = lane + 32;
            }
        }
        if (score_groups) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (lane + 32 * j < P.E)
                    rank_val[lane + 32 * j + (((lane + 32 * j) * P.size_inv) >> 20)] = lg[j] + 0.f;
        }
        __syncwarp();
    }
    int my_e = 0;
    {
        const int live = grouped ? (P.topk_group * P.size + 31) >> 5 : (P.E + 31) >> 5;  // candidates per lane
        const auto run = [&](auto n) {
            return pick_rounds<EPL, decltype(n)::value>(P, bias, sc, lane, grouped, tol_rel, tol_abs, lmax, lg, full,
                                                          val_is_logit);
        };
        if (EPL == 1 || live == 1) my_e = run(Int<1>{});
        else if (EPL == 2 || live == 2) my_e = run(Int<(EPL < 2 ? EPL : 2)>{});
        else if (EPL == 4 || live <= 4) my_e = run(Int<(EPL < 4 ? EPL : 4)>{});
        else if (EPL == 8 || live <= 8) my_e = run(Int<(EPL < 8 ? EPL : 8)>{});
        else my_e = run(Int<EPL>{});
    }
    if (full) {
        my_e = pick_fp64<EPL>(P, bias, lmax, sc, lane);
    }
    float w = 0.f;
    if (lane < P.k) {
        w = sc->val[my_e];
        if (val_is_logit) w = w == -INFINITY ? 0.f : score32(P.scoring, w, lmax, inv_z);
    }
    if (P.renorm) {
        float den = w;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            if (o < P.k) den += __shfl_xor_sync(0xffffffffu, den, o);  // lanes from k on hold 0
        // Underflow takes up to 2^-75 of a score (2^-126 where no root follows): nothing of a sum above 2^-50, but of a
        // smaller one what fp32 could tell, down to all of it (every pick's logit below -87, or as far below the largest)
        if (__shfl_sync(0xffffffffu, den, 0) >= 0x1p-50f) w = __fdividef(w, den);
        else w = weight_fp64(P.scoring, lane < P.k ? logits[my_e] : 0.f, lmax, lane < P.k);
    }
    if (lane < P.k) {
        ids[lane] = my_e;
        wout[lane] = w * P.scaling;
    }
    __syncwarp();  // the scratch is the next token's
}

// ------------------------------------------------------------------------------------------
// From logits in memory: one warp per token.
// ------------------------------------------------------------------------------------------
template <int EPL>
constexpr int given_warps() { return EPL == 16 ? 4 : 8; }

template <int EPL>
__global__ void __launch_bounds__(given_warps<EPL>() * 32)
topk_grouped_kernel(const float* __restrict__ logits, const float* __restrict__ bias, int T,
                    const __grid_constant__ GroupRule P,
                    int32_t* __restrict__ ids, float* __restrict__ wout, int32_t* __restrict__ status) {
    __shared__ RouteScratch<EPL> scratch[given_warps<EPL>()];
    pdl_wait();  // logits come from the router kernel
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * given_warps<EPL>() + warp;
    if (t >= T) return;
    const float* row = logits + t * P.E;
    float raw[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) raw[j] = lane + 32 * j < P.E ? __ldcg(row + lane + 32 * j) : 0.f;
    float bv[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) bv[j] = bias && lane + 32 * j < P.E ? bias[lane + 32 * j] : 0.f;
    route_token<EPL>(P, raw, bv, row, bias, &scratch[warp], lane, ids + t * P.k, wout + t * P.k, status);
}

template <int EPL>
cudaError_t launch_given(const float* logits, const float* bias, int T, const GroupRule& P, int32_t* ids,
                         float* w, int32_t* status, cudaStream_t st) {
    constexpr int W = given_warps<EPL>();
    return launch_pdl(topk_grouped_kernel<EPL>, dim3((unsigned)(((int64_t)T + W - 1) / W)), dim3(32 * W), st,
                      logits, bias, T, P, ids, w, status);
}

// ------------------------------------------------------------------------------------------
// From tokens: the router product and the selection in one launch, for E <= 256.  More experts go through
// the same kernel in blocks of up to 256 (grid y) that write their logits only; the selection follows.
//
// A cluster takes 128 tokens, its CTAs a part of K each: x (the MMA's 128 rows) and the router (all
// experts as the N side) stream through a TMA ring into a TMEM accumulator.  Each CTA owns
// 128 / splits of the tokens; the partial logits go from tensor memory to the owners' shared memory,
// where a warp per token adds them in rank order, writes the logits and selects.  The logits never
// come back from memory, and for few tokens a launch is saved.  Where K has fewer stages than there is
// room for CTAs, the CTAs beyond add no part and only own tokens (178 x 72 x 160: 15.9 us with 2 CTAs a
// tile, 8.1 with 16).
// ------------------------------------------------------------------------------------------
struct FusedMaps {
    CUtensorMap x, w;
};

struct FusedArgs {
    int T;
    int E;                  // all experts, the length of a row of logits
    int select;             // 0: write the logits only
    FusedPlan p;
    const float* bias;
    float* logits;
    int32_t* ids;
    float* w;
    int32_t* status;
};

template <int EPL>
__global__ void __launch_bounds__(kFusedThreads, 1)
route_fused_kernel(const __grid_constant__ FusedMaps maps, const __grid_constant__ FusedArgs a,
                   const __grid_constant__ GroupRule P) {
    using namespace tc;
    extern __shared__ uint8_t rf_smem[];
    __shared__ uint64_t full[kFusedStagesMax], empty[kFusedStagesMax], acc_full;
    __shared__ uint32_t tmem_slot;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(rf_smem) + 1023) & ~uintptr_t(1023));
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int splits = (int)cluster_size(), rank = (int)cluster_rank();
    const int64_t t0 = (int64_t)(blockIdx.x / splits) * 128;
    const int rows = (int)min((int64_t)128, a.T - t0);  // tokens of this tile
    const int stage_bytes = kFusedA + a.p.n * 128;
    const int k_begin = a.p.nk * rank / a.p.parts, k_end = a.p.nk * (rank + 1) / a.p.parts;  // nk < 2^26, rank < 16
    const int steps = rank < a.p.parts ? k_end - k_begin : 0;
    const int e0 = (int)blockIdx.y * a.p.n, experts = min(a.p.n, a.E - e0);  // of this block
    const int pitch = a.p.n + 4;  // floats: 16-byte accesses of eight rows meet 32 banks
    float* landing = reinterpret_cast<float*>(smem + a.p.landing_at);  // [rank][own token][pitch]
    const uint32_t tm_cols = (uint32_t)tmem_columns(a.p.n);
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        fence_mbar_init();
        prefetch_tmap(&maps.x);
        prefetch_tmap(&maps.w);
    }
    if (warp == 1) tmem_alloc(&tmem_slot, tm_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    cluster_arrive();  // this CTA runs: its shared memory may be written from the others
    pdl_wait();
    pdl_trigger();  // after the allocation, so that a waiting successor cannot hold the columns
    auto give_up = [&]() { status_or(a.status, MOE_DEV_TIMEOUT); };
    // the rest of an elected lane's warp waits at the end of its role (linear.cu says why)
    if (warp == 0) {
        if (elect_one()) {  // TMA producer
            const uint32_t bytes = (uint32_t)(a.p.box_x * 128 + a.p.n * 128);
            int issued = 0;
            RingPos at;
            for (int i = 0; i < steps; ++i, at.next(a.p.stages)) {
                const int s = at.slot;
                if (!mbar_wait_suspended(&empty[s], at.parity ^ 1)) {
                    give_up();
                    break;
                }
                uint8_t* base = smem + s * stage_bytes;
                const int kx = (k_begin + i) * kFusedK;
                mbar_arrive_expect_tx(&full[s], bytes);
                tma_load_2d(base + kFusedA, &maps.w, kx, e0, &full[s]);
                tma_load_2d(base, &maps.x, kx, (int)t0, &full[s]);  // rows beyond the box: never read back
                ++issued;
            }
            // whoever gives up, no copy is in flight when the CTA ends
            for (int i = issued < a.p.stages ? issued : a.p.stages; i > 0; --i) {
                at.back(a.p.stages);
                mbar_wait_suspended(&full[at.slot], at.parity);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {  // MMA issuer
            const uint32_t idesc = idesc_bf16(128, a.p.n);
            RingPos at;
            for (int i = 0; i < steps; ++i, at.next(a.p.stages)) {
                const int s = at.slot;
                if (!mbar_wait_suspended(&full[s], at.parity)) {
                    give_up();
                    break;
                }
                tc_fence_after();
                const uint64_t ad = smem_desc(smem_u32(smem + s * stage_bytes), 16, 1024, kLayoutSw128);
#pragma unroll
                for (int j = 0; j < 4; ++j)  // K 16 per MMA: 32 bytes (two units) along the swizzled row
                    tc_mma_bf16(tmem, ad + 2 * j, ad + (kFusedA >> 4) + 2 * j, idesc, (i | j) != 0);
                tc_commit(&empty[s]);
            }
            tc_commit(&acc_full);  // arrives when every MMA has completed
            if (!mbar_wait_suspended(&acc_full, 0)) give_up();
            tc_fence_before();
        }
        __syncwarp();
    }
    __syncthreads();  // all wait here for that: a barrier, not polls, beside the threads that feed the MMAs
    cluster_wait();
    if (a.p.landing_at == 0) cluster_sync();  // over the ring: no CTA's copies or MMAs may still use it
    {  // a warp's lane quarter: tokens 32 q + lane; the four warps of a quarter share the experts
        tc_fence_after();
        const int q = warp & 3, row = 32 * q + lane;
        if (32 * q < rows && rank < a.p.parts) {
            const int owner = min(row / a.p.own, splits - 1), at = row - owner * a.p.own;
            const uint32_t dst = map_rank(smem_u32(landing + ((int64_t)rank * a.p.own + at) * pitch), owner);
            for (int c = 16 * (warp >> 2); c < a.p.n; c += 16 * (kFusedThreads / 128)) {
                uint32_t v[16];
                tmem_ld_16(tmem + ((uint32_t)(32 * q) << 16) + c, v);
                tmem_ld_wait();
                if (row < rows)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        st_cluster_v4(dst + (c + i) * 4, v[i], v[i + 1], v[i + 2], v[i + 3]);
                __syncwarp();
            }
        }
        tc_fence_before();
    }
    float bv[EPL];  // on its way while the parts land
#pragma unroll
    for (int j = 0; j < EPL; ++j) bv[j] = a.bias && lane + 32 * j < experts ? a.bias[lane + 32 * j] : 0.f;
    __syncthreads();
    cluster_sync();  // every part has landed
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, tm_cols);
    }
    auto* scratch = reinterpret_cast<RouteScratch<EPL>*>(smem + a.p.scratch_at) + warp;
    const int mine = min(a.p.own, rows - rank * a.p.own);  // tokens of this CTA (may be negative)
    for (int i = warp; i < mine; i += kFusedThreads / 32) {
        const int64_t t = t0 + (int64_t)rank * a.p.own + i;
        float raw[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) raw[j] = 0.f;
#pragma unroll 2
        for (int s = 0; s < a.p.parts; ++s) {
            const float* src = landing + ((int64_t)s * a.p.own + i) * pitch + lane;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (lane + 32 * j < experts) raw[j] += src[32 * j];
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (lane + 32 * j < experts) a.logits[t * a.E + e0 + lane + 32 * j] = raw[j];
        if (a.select)
            route_token<EPL>(P, raw, bv, a.logits + t * a.E, a.bias, scratch, lane, a.ids + t * P.k, a.w + t * P.k, a.status);
    }
}

template <int EPL>
cudaError_t launch_fused(const FusedMaps& m, const FusedArgs& a, const GroupRule& P, cudaStream_t st) {
    const auto kernel = route_fused_kernel<EPL>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t err = allow_large_launch(kernel, kCtaSmemMax, allowed);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)a.T + 127) / 128 * a.p.splits), (unsigned)a.p.blocks);
    cfg.blockDim = dim3(kFusedThreads);
    cfg.dynamicSmemBytes = a.p.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.p.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, m, a, P);
}

GroupRule make_rule(const float* bias, int E, int k, int scoring, int renorm, float scaling, int n_group,
                    int topk_group, int group_top) {
    const int size = E / n_group;
    int shift = 0;
    while ((2 << shift) * n_group <= 32) ++shift;
    return GroupRule{E, k, scoring, renorm, n_group, topk_group, group_top, bias == nullptr, size,
                     ((1 << 20) + size - 1) / size, 1 << shift, shift, scaling};
}

}  // namespace

cudaError_t launch_topk_grouped(const float* logits, const float* bias, int T, int E, int k, int scoring,
                                int renorm, float scaling, int n_group, int topk_group, int group_top,
                                int32_t* ids, float* w, int32_t* status, cudaStream_t st) {
    const GroupRule P = make_rule(bias, E, k, scoring, renorm, scaling, n_group, topk_group, group_top);
    if (E <= 32) return launch_given<1>(logits, bias, T, P, ids, w, status, st);
    if (E <= 64) return launch_given<2>(logits, bias, T, P, ids, w, status, st);
    if (E <= 128) return launch_given<4>(logits, bias, T, P, ids, w, status, st);
    if (E <= 256) return launch_given<8>(logits, bias, T, P, ids, w, status, st);
    return launch_given<16>(logits, bias, T, P, ids, w, status, st);
}

cudaError_t launch_route_fused(const void* x, const void* wr, const float* bias, int T, int E, int H, int k,
                               int scoring, int renorm, float scaling, int n_group, int topk_group,
                               int group_top, float* logits, int32_t* ids, float* w, int32_t* status,
                               cudaStream_t st) {
    const GroupRule P = make_rule(bias, E, k, scoring, renorm, scaling, n_group, topk_group, group_top);
    FusedArgs a{};
    if (!plan_fused(T, E, H, a.p)) return cudaErrorNotSupported;
    a.T = T;
    a.E = E;
    a.select = a.p.blocks == 1;
    a.bias = a.select ? bias : nullptr;
    a.logits = logits; a.ids = ids; a.w = w; a.status = status;
    FusedMaps m{};
    if (!encode_rows16(&m.x, x, H, T, H, a.p.box_x, 64) || !encode_rows16(&m.w, wr, H, E, H, a.p.n, 64))
        return cudaErrorNotSupported;
    if (E <= 32) return launch_fused<1>(m, a, P, st);
    if (E <= 64) return launch_fused<2>(m, a, P, st);
    if (E <= 128) return launch_fused<4>(m, a, P, st);
    const cudaError_t err = launch_fused<8>(m, a, P, st);
    if (err != cudaSuccess || a.select) return err;
    return launch_topk_grouped(logits, bias, T, E, k, scoring, renorm, scaling, n_group, topk_group, group_top, ids, w,
                               status, st);
}

}  // namespace moe
