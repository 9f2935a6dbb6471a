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
// where a comparison that decides the result falls inside the bound, the token's selection runs
// again in fp64.  Without a bias every score grows with its logit, and experts are ranked by
// the logits themselves, which needs no bound.
#include "common.cuh"
#include "kernels.h"
#include "topk.cuh"

namespace moe {

namespace {

constexpr int kRgWarps = 8;  // tokens per CTA

template <typename R>
__device__ __forceinline__ R score_of(int scoring, R l, R lmax, R zall) {
    if (l == -INFINITY) return R(0);
    if (scoring == MOE_SCORE_SOFTMAX || scoring == MOE_SCORE_SOFTMAX_BIAS) return exp(l - lmax) / zall;
    if (scoring == MOE_SCORE_SQRTSOFTPLUS) return sqrt(l > R(40) ? l : log1p(exp(l)));
    return R(1) / (R(1) + exp(-l));
}

struct GroupRule {
    int E, k, scoring, renorm, n_group, topk_group, group_top, by_logit;
    float scaling;
};

// Relative error bound of an fp32 selection score: expf, the additions and the division are
// within 2^-22 of |s|; a softmax denominator summed over 512 logits adds up to 2^-19.7.
__device__ __forceinline__ float score_eps(int scoring) {
    return scoring == MOE_SCORE_SOFTMAX || scoring == MOE_SCORE_SOFTMAX_BIAS ? 0x1p-19f : 0x1p-21f;
}

// One warp selects one token's experts, in R = float or double.  lg: the lane's logits (-inf for
// a non-finite one or beyond E), bv: their biases; sm: E values of scratch.  On return lane j < k
// holds pick j.  The result says (float only) whether a comparison fell inside the error bound.
template <int EPL, typename R>
__device__ __forceinline__ bool select_grouped(const GroupRule& P, const float (&lg)[EPL],
                                               const float (&bv)[EPL], float lmax32, R* sm, int lane,
                                               int& my_e) {
    constexpr bool kFloat = sizeof(R) == 4;
    const bool softmax = P.scoring == MOE_SCORE_SOFTMAX || P.scoring == MOE_SCORE_SOFTMAX_BIAS;
    const bool need_score = !P.by_logit || P.group_top == 2;
    const R lmax = lmax32;
    R v[EPL];    // ranks the experts
    R zall = 1;
    if (need_score && softmax) {
        zall = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) zall += lg[j] == -INFINITY ? R(0) : exp(R(lg[j]) - lmax);
#pragma unroll
        for (int o = 16; o; o >>= 1) zall += __shfl_xor_sync(0xffffffffu, zall, o);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + 32 * j;
        R s = -INFINITY;
        v[j] = -INFINITY;
        if (e < P.E && lg[j] != -INFINITY) {
            if (need_score) s = score_of<R>(P.scoring, R(lg[j]), lmax, zall);
            // a bias that is not finite ranks its expert last
            v[j] = P.by_logit ? R(lg[j]) : (isfinite(bv[j]) ? s + R(bv[j]) : R(-INFINITY));
        }
        // what the groups add up: the ranking value, or with two per group the scores
        if (e < P.E) sm[e] = P.by_logit && P.group_top == 2 ? s : v[j];
    }
    __syncwarp();
    const R smax = kFloat && need_score ? score_of<R>(P.scoring, lmax, lmax, zall) : R(0);
    const R eps = kFloat ? R(score_eps(P.scoring)) : R(0);
    bool close = false;

    // group scores: 32 / n_group lanes (a power of two) share a group; lanes of sub-index 0 keep
    // the score of groups lane / per and, above 32 groups, + 32
    const int size = P.E / P.n_group;
    int per = 1;
    while (per * 2 * P.n_group <= 32) per *= 2;
    unsigned long long kept = ~0ull;
    if (P.topk_group < P.n_group) {
        R gs[2], tol[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int g = lane / per + 32 * q;
            R m1 = -INFINITY, m2 = -INFINITY;
            if (g < P.n_group) {
                for (int i = lane % per; i < size; i += per) {
                    const R x = sm[g * size + i];
                    m2 = x > m1 ? m1 : (x > m2 ? x : m2);
                    m1 = x > m1 ? x : m1;
                }
            }
            for (int o = per / 2; o; o >>= 1) {
                const R b1 = __shfl_xor_sync(0xffffffffu, m1, o);
                const R b2 = __shfl_xor_sync(0xffffffffu, m2, o);
                const R lo = m1 < b1 ? m1 : b1;
                const R hi2 = m1 > b1 ? m2 : b2;
                m1 = m1 > b1 ? m1 : b1;
                m2 = lo > hi2 ? lo : hi2;
            }
            gs[q] = P.group_top == 2 ? m1 + m2 : m1;
            tol[q] = !need_score ? R(0)
                                 : eps * (fabs(m1) + (P.group_top == 2 ? fabs(m2) : R(0)) + 4 * smax);
        }
        // rank of each group among all: the kept ones are those with rank < topk_group
        kept = 0;
        for (int g = 0; g < P.n_group; ++g) {
            const R mine = __shfl_sync(0xffffffffu, g < 32 ? gs[0] : gs[1], (g & 31) * per);
            // groups above 32 come only with per == 1, so lane l holds groups l and l + 32
            bool ahead0 = false, ahead1 = false, amb = false;
            const R mtol = kFloat ? __shfl_sync(0xffffffffu, g < 32 ? tol[0] : tol[1], (g & 31) * per) : R(0);
            const bool judge = kFloat && need_score && mine > -INFINITY;
            const int g0 = lane / per;
            if (lane % per == 0 && g0 < P.n_group && g0 != g) {
                ahead0 = gs[0] > mine || (gs[0] == mine && g0 < g);
                amb = judge && gs[0] > -INFINITY && fabs(gs[0] - mine) <= tol[0] + mtol;
            }
            if (g0 + 32 < P.n_group && per == 1 && g0 + 32 != g) {
                ahead1 = gs[1] > mine || (gs[1] == mine && g0 + 32 < g);
                amb = amb || (judge && gs[1] > -INFINITY && fabs(gs[1] - mine) <= tol[1] + mtol);
            }
            const unsigned b0 = __ballot_sync(0xffffffffu, ahead0);
            const unsigned b1 = __ballot_sync(0xffffffffu, ahead1);
            const int rank = __popc(b0) + __popc(b1);
            if (rank < P.topk_group) kept |= 1ull << g;
            // only the border between kept and dropped matters
            if (kFloat && (rank == P.topk_group - 1 || rank == P.topk_group))
                close = close || __any_sync(0xffffffffu, amb);
        }
    }

#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + 32 * j;
        if (e >= P.E || !((kept >> (e / size)) & 1)) v[j] = NAN;  // never picked
    }
    my_e = 0;
    R prev = INFINITY;
    for (int r = 0; r < P.k; ++r) {
        R best = -INFINITY;
        int be = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 32 * j;
            if (v[j] > best || (v[j] == best && e < be)) {
                best = v[j];
                be = e;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const R ob = __shfl_xor_sync(0xffffffffu, best, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (ob > best || (ob == best && oe < be)) {
                best = ob;
                be = oe;
            }
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (lane + 32 * j == be) v[j] = NAN;
        if (lane == r) my_e = be;
        if (kFloat && !P.by_logit && best > -INFINITY)
            close = close || prev - best <= 2 * eps * (fabs(best) + 2 * smax);
        prev = best;
    }
    if (kFloat && !P.by_logit && prev > -INFINITY) {  // the best of those left behind
        bool amb = false;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            amb = amb || (v[j] > -INFINITY && prev - v[j] <= 2 * eps * (fabs(prev) + 2 * smax));
        close = close || __any_sync(0xffffffffu, amb);
    }
    return close;
}

template <int EPL>
__global__ void __launch_bounds__(kRgWarps * 32)
topk_grouped_kernel(const float* __restrict__ logits, const float* __restrict__ bias, int T, GroupRule P,
                    int32_t* __restrict__ ids, float* __restrict__ wout, int32_t* __restrict__ status) {
    extern __shared__ double rg_smem[];
    pdl_wait();  // logits come from the router kernel
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kRgWarps + warp;
    if (t >= T) return;
    double* sm = rg_smem + warp * P.E;
    const float* row = logits + (size_t)t * P.E;
    float lg[EPL], bv[EPL];
    float lmax = -INFINITY;
    bool nonfinite = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = lane + 32 * j;
        lg[j] = e < P.E ? row[e] : -INFINITY;
        bv[j] = bias && e < P.E ? bias[e] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        if (lane + 32 * j < P.E && !isfinite(lg[j])) {
            nonfinite = true;
            lg[j] = -INFINITY;
        }
        lmax = fmaxf(lmax, lg[j]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
    if (__any_sync(0xffffffffu, nonfinite) && lane == 0) status_or(status, MOE_DEV_NONFINITE);

    int e;
    if (select_grouped<EPL, float>(P, lg, bv, lmax, reinterpret_cast<float*>(sm), lane, e))
        select_grouped<EPL, double>(P, lg, bv, lmax, sm, lane, e);

    // weights of the picks
    const bool softmax = P.scoring == MOE_SCORE_SOFTMAX || P.scoring == MOE_SCORE_SOFTMAX_BIAS;
    float z = 1.f;
    if (softmax && !P.renorm) {
        z = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) z += lg[j] == -INFINITY ? 0.f : expf(lg[j] - lmax);
#pragma unroll
        for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    float s = 0.f;
    if (lane < P.k) {
        const float l = row[e];
        s = isfinite(l) ? score_of<float>(P.scoring, l, lmax, z) : 0.f;
    }
    if (P.renorm) {
        float den = s;
#pragma unroll
        for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
        s = den > 0.f ? s / den : 0.f;
    }
    if (lane < P.k) {
        ids[(size_t)t * P.k + lane] = e;
        wout[(size_t)t * P.k + lane] = s * P.scaling;
    }
}

template <int EPL>
cudaError_t launch_epl(const float* logits, const float* bias, int T, const GroupRule& P, int32_t* ids,
                       float* w, int32_t* status, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((T + kRgWarps - 1) / kRgWarps);
    cfg.blockDim = dim3(kRgWarps * 32);
    cfg.dynamicSmemBytes = sizeof(double) * kRgWarps * P.E;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, topk_grouped_kernel<EPL>, logits, bias, T, P, ids, w, status);
}

}  // namespace

cudaError_t launch_topk_grouped(const float* logits, const float* bias, int T, int E, int k, int scoring,
                                int renorm, float scaling, int n_group, int topk_group, int group_top,
                                int32_t* ids, float* w, int32_t* status, cudaStream_t st) {
    const GroupRule P{E, k, scoring, renorm, n_group, topk_group, group_top, bias == nullptr, scaling};
    if (E <= 32) return launch_epl<1>(logits, bias, T, P, ids, w, status, st);
    if (E <= 64) return launch_epl<2>(logits, bias, T, P, ids, w, status, st);
    if (E <= 128) return launch_epl<4>(logits, bias, T, P, ids, w, status, st);
    if (E <= 256) return launch_epl<8>(logits, bias, T, P, ids, w, status, st);
    return launch_epl<16>(logits, bias, T, P, ids, w, status, st);
}

}  // namespace moe
