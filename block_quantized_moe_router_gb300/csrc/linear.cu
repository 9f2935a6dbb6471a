// linear.cu -- y = f(x W^T + b) [* (x V^T + c)] [+ r], fp32 sums, one rounding.
//
// Two kernels on tcgen05.mma.kind::f16, both fed by TMA (boxes of 64 elements of K, 128-byte swizzled
// rows; what lies beyond a matrix reads as zero) into accumulators in tensor memory:
//
//   linear_few_kernel   few rows.  The time is that of streaming the weights, so the weights are
//       the MMA's 128-row operand and the rows of x its N side (16 to 128 columns): each weight
//       byte passes through shared memory once, however few rows there are.  K is split over the
//       CTAs of a cluster so that a narrow matrix still occupies the SMs; the partial sums meet
//       through distributed shared memory, added in rank order (equal calls give equal bits).
//   linear_many_kernel  many rows.  CTA pairs (cta_group::2) compute 256 x up to 256 tiles: each
//       CTA stages its own 128 rows of x and half of the weight rows, so the pair reads each
//       operand byte once for both.  Persistent over the tiles, two accumulators in TMEM, so the
//       epilogue of one tile runs under the MMAs of the next.
//
// The gated form takes its weight rows half from W and half from V, so z and its factor meet in one
// accumulator and neither goes through memory.  Every wait is bounded: one that gives up sets
// MOE_DEV_TIMEOUT and the CTA winds down.
#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch_plan.h"
#include "tc_ptx.cuh"

#include <type_traits>

namespace moe {

namespace {

using namespace tc;

constexpr int kLinA = 128 * 128;                // bytes of a 128-row operand stage

struct LinMaps {
    CUtensorMap x, w, v, res, out;
};

struct LinArgs {
    int T, N, nk;       // nk: stages of K in all
    int func, gated, f16;
    int rows_t, stages; // few rows: rows of x per tile, stages of the ring
    int tma_rows;       // many rows: out and the residual go by TMA
    int width;          // many rows: rows of weights per tile
    int64_t ldr, ldo;
    const float *bias, *bias_mul;
    const void* res;
    void* out;
    int32_t* status;
};

// ---- CTA-pair primitives -------------------------------------------------------------------------
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// TMA load of a CTA pair: the bytes land here, the count on the mapped barrier of either CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* m, int x, int y,
                                              uint32_t mapped_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(mapped_bar)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrive on `bar` of the CTAs in `mask` (both of the pair) once this thread's earlier MMAs have completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar, uint32_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)), "h"((uint16_t)mask) : "memory");
}
template <int PAIR>
__device__ __forceinline__ void mma_f16kind(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(ad), "l"(bd),
            "r"(idesc), "r"(acc) : "memory");
    else
        tc_mma_bf16(d, ad, bd, idesc, acc);
}
// kind::f16: fp32 D, A and B both bf16 (format 1) or both f16 (format 0), K-major.
__device__ __forceinline__ uint32_t idesc_f16kind(uint32_t M, uint32_t N, bool f16) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// ---- epilogue arithmetic -------------------------------------------------------------------------
// The function over C values: one branch for all of them (a branch per value, unrolled, costs more
// in instruction fetch than the arithmetic).  __fdividef is off by 2 units of the last place of fp32, and 0
// where the divisor passes 2^126, where the result is below 2^-119; the exact division has a branch of its
// own per value (8192 x 4096 x 1024 with SiLU: 86 us, 53 so, 51 without a function).
template <int C>
__device__ __forceinline__ void apply_func(int func, float (&z)[C]) {
    switch (func) {
        case MOE_FUNC_SILU:
#pragma unroll
            for (int i = 0; i < C; ++i) z[i] = __fdividef(z[i], 1.f + __expf(-z[i]));
            break;
        case MOE_FUNC_GELU:
#pragma unroll
            for (int i = 0; i < C; ++i) z[i] = 0.5f * z[i] * (1.f + erff(z[i] * 0.70710678f));
            break;
        case MOE_FUNC_GELU_TANH:  // 0.5 (1 + tanh u) = sigmoid(2 u)
#pragma unroll
            for (int i = 0; i < C; ++i)
                z[i] = __fdividef(z[i], 1.f + __expf(-1.5957691f * (z[i] + 0.044715f * z[i] * z[i] * z[i])));
            break;
        case MOE_FUNC_RELU:  // not fmaxf: a NaN stays
#pragma unroll
            for (int i = 0; i < C; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];
            break;
    }
}
// z += the C 16-bit values packed in w.
template <int C>
__device__ __forceinline__ void add_packed(float (&z)[C], const uint32_t (&w)[C / 2], bool f16) {
    if (f16) {
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            z[2 * i] += f.x;
            z[2 * i + 1] += f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            z[2 * i] += __uint_as_float(w[i] << 16);
            z[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}
template <int C>
__device__ __forceinline__ void pack_all(const float (&z)[C], uint32_t (&w)[C / 2], bool f16) {
    if (f16) {
#pragma unroll
        for (int i = 0; i < C / 2; ++i)
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(z[2 * i + 1]), "f"(z[2 * i]));
    } else {
#pragma unroll
        for (int i = 0; i < C / 2; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(z[2 * i + 1]), "f"(z[2 * i]));
    }
}

// The residual of feature n of up to C consecutive rows from t on, and these rows' results (the lanes of a
// warp hold consecutive features).
template <int C>
__device__ __forceinline__ void load_residual(const LinArgs& a, int64_t t, int rows, int n, uint32_t (&rw)[C]) {
    const uint16_t* res = static_cast<const uint16_t*>(a.res) + t * a.ldr + n;
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (i < rows) rw[i] = res[i * a.ldr];
}
template <int C>
__device__ __forceinline__ void finish_feature(const LinArgs& a, int64_t t, int rows, int n, float (&z)[C],
                                               const float (&u)[C], const uint32_t (&rw)[C]) {
    const float b = a.bias ? __ldg(a.bias + n) : 0.f, c = a.bias_mul ? __ldg(a.bias_mul + n) : 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) z[i] += b;
    apply_func(a.func, z);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        if (a.gated) z[i] *= u[i] + c;
        if (a.res) z[i] += a.f16 ? __half2float(__ushort_as_half((unsigned short)rw[i])) : __uint_as_float(rw[i] << 16);
    }
    uint32_t w[C / 2];
    pack_all(z, w, a.f16);
    uint16_t* out = static_cast<uint16_t*>(a.out) + t * a.ldo + n;
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (i < rows) out[i * a.ldo] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
}

// 16 outputs of one row, biases in shared memory, the residual's 16 values packed in rw (zeros
// without one), to packed results.
__device__ __forceinline__ void combine16(const LinArgs& a, const float* bias, const float* bias_mul,
                                          float (&z)[16], const float (&u)[16], const uint32_t (&rw)[8],
                                          uint32_t (&ow)[8]) {
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 b = *reinterpret_cast<const float4*>(bias + i);
            z[i] += b.x; z[i + 1] += b.y; z[i + 2] += b.z; z[i + 3] += b.w;
        }
    }
    apply_func(a.func, z);
    if (a.bias_mul) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 b = *reinterpret_cast<const float4*>(bias_mul + i);
            z[i] *= u[i] + b.x; z[i + 1] *= u[i + 1] + b.y; z[i + 2] *= u[i + 2] + b.z; z[i + 3] *= u[i + 3] + b.w;
        }
    } else if (a.gated) {
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] *= u[i];
    }
    if (a.res) add_packed(z, rw, a.f16);
    pack_all(z, ow, a.f16);
}

// Whether rows of `p` (ld elements apart) all start at multiples of `bytes`.
inline bool rows_aligned(const void* p, int64_t ld, int bytes) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(2 * ld)) & (uintptr_t)(bytes - 1)) == 0;
}

// ------------------------------------------------------------------------------------------
// Few rows.  grid (tiles of W rows * CTAs of a cluster, tiles of x rows).  A tile is 128 rows of W, or 64 of
// W and 64 of V; `splits` parts of K make its cluster.  Warp 0 loads, warp 1 issues the MMAs, and the eight
// warps send the accumulator (lane = W row, column = row of x) to its owners: each CTA owns `own` columns of
// its features and has a landing area for every part of them.  After one cluster barrier each CTA adds its
// columns' parts, in rank order, from its own shared memory.  Where a tile has one part of K and no gate, a lane
// has all of its feature and the rows go out straight from tensor memory (pairs, 128 rows of 7168 x 2048: 11.8
// us, 14.3 through the landing area).
//
// PAIR: a part of K belongs to two CTAs (cta_group::2), each with half of the tile's weight rows and half of
// the rows of x, which both use.  An SM's share of the L2 rate bounds the loads, and of every 64 elements of
// K a CTA then takes 64 (rows of W) + rows / 2 lines and not 128 + rows; its accumulator, and with it the
// exchange, is half as large.  In tensor memory lanes 0 to 63 hold the CTA's 64 weight rows against the first
// half of x, lanes 64 to 127 against the second.  128 rows of 7168 x 2048: 11.8 us against 15.7 in single CTAs;
// 16 rows 9.9 against 8.8, where the latency of a stage counts and not its bytes.
// ------------------------------------------------------------------------------------------
constexpr int kFewThreads = 256;

template <bool PAIR>
__global__ void __launch_bounds__(kFewThreads, 4)
linear_few_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinArgs a) {
    using F = Few<PAIR>;
    extern __shared__ uint8_t lin_smem[];
    __shared__ uint64_t full[kFewStages], empty[kFewStages], acc_full;
    __shared__ uint32_t tmem_slot;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_smem) + 1023) & ~uintptr_t(1023));
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const uint32_t ctas = cluster_size(), cta = cluster_rank();
    const uint32_t splits = ctas / F::kCtas, rank = cta / F::kCtas;  // part of K
    const uint32_t half = cta % F::kCtas, first = cta - half;        // CTA of the pair, and its first one
    const int per_cta = a.gated ? F::kW / 2 : F::kW;                 // features
    const int n0 = ((int)(blockIdx.x / ctas) * F::kCtas + (int)half) * per_cta;
    const int t0 = (int)blockIdx.y * a.rows_t;
    const int NT = a.rows_t, x_rows = NT / F::kCtas;  // of the tile, and of them here
    const int k_begin = (int)((uint32_t)a.nk * rank / splits), k_end = (int)((uint32_t)a.nk * (rank + 1) / splits);  // nk < 2^15
    const int stage_bytes = F::stage(NT);
    const int ncols = min(NT, a.T - t0);
    // [rank][W row][own columns, padded so that 16-byte accesses of 8 rows meet 32 banks]
    float* landing = reinterpret_cast<float*>(smem + a.stages * stage_bytes);
    const int own = F::own(NT, (int)splits), pitch = F::pitch(own);
    const uint32_t tm_cols = (uint32_t)F::columns(NT);
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        fence_mbar_init();
        prefetch_tmap(&maps.x);
        prefetch_tmap(&maps.w);
        if (a.gated) prefetch_tmap(&maps.v);
    }
    if (warp == 1) {
        if constexpr (PAIR) tmem_alloc_pair(&tmem_slot, tm_cols);
        else tmem_alloc(&tmem_slot, tm_cols);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // This CTA runs: its shared memory may be written from the others.  A pair signals each other's barriers
    // from the first stage on, single CTAs meet at the exchange.
    cluster_arrive();
    if constexpr (PAIR) cluster_wait();
    pdl_wait();
    pdl_trigger();  // after the allocation, so that a waiting successor cannot hold the columns
    auto give_up = [&]() { status_or(a.status, MOE_DEV_TIMEOUT); };
    const int my_c0 = (int)rank * own, my_cols = min(own, ncols - my_c0);  // this CTA's columns
    const bool direct = splits == 1 && !a.gated;  // a lane has all of its feature: nothing to exchange
    const int steps = k_end - k_begin;
    // The elected lane's role is all that its warp does until the lane is done: the rest of the warp waits at the end of
    // the role, so that nothing it might run shares the warp's uniform registers with the lane's copies and MMAs
    if (warp == 0) {
        if (elect_one()) {
            const uint32_t full0 = PAIR ? map_rank(smem_u32(&full[0]), first) : smem_u32(&full[0]);
            int issued = 0;
            RingPos at;
            for (int i = 0; i < steps; ++i, at.next(a.stages)) {
                const int s = at.slot;
                if (!mbar_wait_suspended(&empty[s], at.parity ^ 1)) {
                    give_up();
                    break;
                }
                uint8_t* base = smem + s * stage_bytes;
                const int kx = (k_begin + i) * kLinK;
                if constexpr (PAIR) {
                    const uint32_t dst = smem_u32(base), bar = full0 + 8 * s;
                    if (half == 0) mbar_arrive_expect_tx(&full[s], 2 * stage_bytes);
                    tma_load_pair(dst, &maps.w, kx, n0, bar);
                    if (a.gated) tma_load_pair(dst + F::kA / 2, &maps.v, kx, n0, bar);
                    tma_load_pair(dst + F::kA, &maps.x, kx, t0 + (int)half * x_rows, bar);
                } else {
                    mbar_arrive_expect_tx(&full[s], stage_bytes);
                    tma_load_2d(base, &maps.w, kx, n0, &full[s]);
                    if (a.gated) tma_load_2d(base + F::kA / 2, &maps.v, kx, n0, &full[s]);
                    tma_load_2d(base + F::kA, &maps.x, kx, t0, &full[s]);
                }
                ++issued;
            }
            // whoever gives up, no copy is in flight when the CTA ends (the pair's arrive at its first CTA)
            if (half == 0)
                for (int i = issued < a.stages ? issued : a.stages; i > 0; --i) {
                    at.back(a.stages);
                    mbar_wait_suspended(&full[at.slot], at.parity);
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            if (half == 0) {
                const uint32_t idesc = idesc_f16kind(128, NT, a.f16);
                RingPos at;
                for (int i = 0; i < steps; ++i, at.next(a.stages)) {
                    const int s = at.slot;
                    if (!mbar_wait_suspended(&full[s], at.parity)) {
                        give_up();
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc(smem_u32(smem + s * stage_bytes), 16, 1024, kLayoutSw128);
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // K 16 per MMA: 32 bytes (two units) along the swizzled row
                        mma_f16kind<PAIR>(tmem, ad + 2 * j, ad + (F::kA >> 4) + 2 * j, idesc, (i | j) != 0);
                    if constexpr (PAIR) tc_commit_pair(&empty[s], 3u << first);
                    else tc_commit(&empty[s]);
                }
                // arrives when every MMA has completed
                if constexpr (PAIR) tc_commit_pair(&acc_full, 3u << first);
                else tc_commit(&acc_full);
            }
            if (!mbar_wait_suspended(&acc_full, 0)) give_up();
            tc_fence_before();
        }
        __syncwarp();
    } else if (warp >= 6) {
        // what the end of the kernel reads comes to L2 while the weights stream: 128-byte lines
        if (a.res)
            for (int i = threadIdx.x - 192; i < my_cols * 2; i += 64) {
                const int n = n0 + 64 * (i & 1);
                if (n < a.N && (i & 1) * 64 < per_cta)
                    prefetch_l2(static_cast<const uint16_t*>(a.res) + ((int64_t)t0 + my_c0 + (i >> 1)) * a.ldr + n);
            }
    }
    __syncthreads();  // all wait here for that: a barrier, not polls, beside the threads that feed the MMAs
    if constexpr (!PAIR) cluster_wait();
    {  // the two warps of a lane quarter take alternate 16 columns
        tc_fence_after();
        const int q = warp & 3;
        const int row = 32 * (PAIR ? q & 1 : q) + lane, c0 = PAIR && q >= 2 ? x_rows : 0;  // of tensor memory column 0
        const uint32_t mine = smem_u32(landing + ((int)rank * F::kW + row) * pitch);
        for (int c = c0 + 16 * (warp >> 2); c < min(ncols, c0 + x_rows); c += 32) {
            if (direct) {
                const int n = n0 + row, rows = min(16, ncols - c);
                uint32_t rw[16] = {};
                if (a.res && n < a.N) load_residual(a, (int64_t)t0 + c, rows, n, rw);
                __syncwarp();  // the read of tensor memory wants the whole warp, N may end inside it
                float z[16];
                tmem_ld_16(tmem + ((uint32_t)(32 * q) << 16) + c - c0, reinterpret_cast<uint32_t(&)[16]>(z));
                tmem_ld_wait();
                if (n < a.N) finish_feature(a, (int64_t)t0 + c, rows, n, z, z, rw);
                __syncwarp();
                continue;
            }
            int owner = c / own, at = c - owner * own;  // of the next four columns
            uint32_t v[16];
            tmem_ld_16(tmem + ((uint32_t)(32 * q) << 16) + c - c0, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (c + i < ncols) {
                    st_cluster_v4(map_rank(mine + at * 4, owner * F::kCtas + half), v[i], v[i + 1], v[i + 2], v[i + 3]);
                    at += 4;
                    if (at == own) {
                        at = 0;
                        ++owner;
                    }
                }
        }
        tc_fence_before();
    }
    // Items of 32 features x 4 rows of x, lane = feature.  The residual is read one item ahead, the first
    // before the parts have landed (the compiler may not: out may be the residual).
    const int blocks = per_cta / 32, shift = blocks >> 1;  // 1, 2 or 4 blocks of features
    const int items = direct ? 0 : ((my_cols + 3) / 4) << shift;
    uint32_t rw[4] = {};
    const auto ahead = [&](int item) {
        const int n = n0 + (item & (blocks - 1)) * 32 + lane, c = (item >> shift) * 4;
        if (a.res && item < items && n < a.N) load_residual(a, (int64_t)t0 + my_c0 + c, min(4, my_cols - c), n, rw);
    };
    ahead(warp);
    cluster_sync();  // every part has landed
    for (int item = warp; item < items; item += kFewThreads / 32) {
        const int r = (item & (blocks - 1)) * 32 + lane, c = (item >> shift) * 4;
        const float* src = landing + r * pitch + c;
        const uint32_t now[4] = {rw[0], rw[1], rw[2], rw[3]};
        ahead(item + kFewThreads / 32);
        float z[4] = {}, u[4] = {};
#pragma unroll
        for (int s = 0; s < kFewSplits / F::kCtas; ++s)
            if (s < (int)splits) {
                const float4 p = *reinterpret_cast<const float4*>(src + s * F::kW * pitch);
                z[0] += p.x; z[1] += p.y; z[2] += p.z; z[3] += p.w;
                if (a.gated) {
                    const float4 g = *reinterpret_cast<const float4*>(src + (s * F::kW + F::kW / 2) * pitch);
                    u[0] += g.x; u[1] += g.y; u[2] += g.z; u[3] += g.w;
                }
            }
        const int n = n0 + r;
        if (n < a.N) finish_feature(a, (int64_t)t0 + my_c0 + c, min(4, my_cols - c), n, z, u, now);
    }
    __syncwarp();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, tm_cols);
        else tmem_dealloc(tmem, tm_cols);
    }
}

// ------------------------------------------------------------------------------------------
// Many rows.  Clusters of two CTAs, one per SM; a pair's tile is 256 rows of x by `width` rows of W
// (gated: width / 2 of W and of V), each CTA holding 128 rows of x and all columns.  Warp 0 loads,
// warp 1 of the pair's first CTA issues the MMAs, warps 2-9 (two per lane quarter, alternate
// columns) turn accumulators into rows and warps 10-13 move rows: the residual comes in and results
// go out through two 16 KB buffers of 64 features (64-byte swizzled halves, so a thread per row
// meets no bank conflicts), a pass of 64 features at a time; the next passes' residual loads
// meanwhile.  Warp 10 alone moves them by TMA; rows that TMA cannot address (not 16-byte aligned) or would
// write beyond (their end is not) are copied by the four warps, a warp's lanes along the row in aligned
// words of two features, which start at the second feature where a row starts off 4 bytes; which rows do is
// a choice made once per pass, so that the copies carry no branch (8192 x 2047 x 2048: 169 us with the epilogue's threads storing their own rows, 58
// feature by feature, 92 with the choice in every row, 49 so, 45 at 2048 features).
//
// A stage is 128 elements of K: with 64 the commit and barrier round trips of twice as many stages
// held the MMAs back (8192^3 without its epilogue 620 us, against 563 with 128, of 574 at the
// measured cuBLAS rate).  Two pairs sharing x by multicast were no faster: clusters of four occupy
// 144 of the 152 SMs.
// ------------------------------------------------------------------------------------------
constexpr int kManyThreads = 448;
constexpr int kManyMovers = 4;
constexpr int kManyStages = 3;
constexpr int kManyHalf = 2 * kLinA;             // 64 elements of K: 128 rows of x, at most 128 of W
constexpr int kManyStageBytes = 2 * kManyHalf;
constexpr int kManySub = 128 * 64;               // bytes of 32 features of 128 rows
constexpr int kManySmem = kManyStages * kManyStageBytes + 4 * kManySub + 1024;
static_assert(columns_covered(kManySmem, kTmemColumns));
constexpr int kManyGroup = 8;  // row tiles that share a pass over the weights

struct ManySched {
    int tiles_t, tiles_n;
    int64_t total;
    __host__ __device__ ManySched(int T, int N, int features) {
        tiles_t = (int)(((int64_t)T + 255) / 256);
        tiles_n = (N + features - 1) / features;
        total = (int64_t)tiles_t * tiles_n;
    }
    // A tile's place: kManyGroup row tiles run through all columns together.  Counted on from tile to tile in 32 bits (a
    // group has fewer than 2^18 tiles): a 64-bit division would be a call, and the thread that issues copies makes none.
    struct Place {
        int64_t tile;
        uint32_t group, rest;
    };
    __device__ __forceinline__ Place begin(int pair) const {
        const uint32_t per = (uint32_t)(kManyGroup * tiles_n);
        return Place{pair, (uint32_t)pair / per, (uint32_t)pair % per};
    }
    __device__ __forceinline__ void next(Place& at, int pairs) const {
        const uint32_t per = (uint32_t)(kManyGroup * tiles_n);
        at.tile += pairs;
        at.rest += (uint32_t)pairs;
        at.group += at.rest / per;
        at.rest %= per;
    }
    // its row tile and column tile
    __device__ __forceinline__ void tiles(const Place& at, int& tt, int& tn) const {
        const uint32_t rows = (uint32_t)min(kManyGroup, tiles_t - (int)at.group * kManyGroup);
        tt = (int)at.group * kManyGroup + (int)(at.rest % rows);
        tn = (int)(at.rest / rows);
    }
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(smem_u32(src)) : "memory");
}

__global__ void __launch_bounds__(kManyThreads, 1)
linear_many_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinArgs a) {
    extern __shared__ uint8_t lin_smem[];
    __shared__ uint64_t full[kManyStages], empty[kManyStages], acc_full[2], acc_empty[2];
    __shared__ uint64_t buf_ready[2], buf_done[2];  // row buffers: usable by the epilogue; written by it
    __shared__ __align__(16) float bias_s[2][128];  // per buffer: 64 of bias, 64 of bias_mul
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_smem) + 1023) & ~uintptr_t(1023));
    uint8_t* rows_s = smem + kManyStages * kManyStageBytes;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const int half = a.width / 2;
    const int per_tile = a.gated ? half : a.width;  // features per tile
    const int subs = per_tile / 32, passes = (per_tile + 63) / 64;
    const bool by_tma = a.tma_rows, res_tma = by_tma && a.res;
    const ManySched sched(a.T, a.N, per_tile);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kManyStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 16);  // the epilogue warps of both CTAs
            mbar_init(&buf_ready[b], by_tma ? 1 : kManyMovers);
            mbar_init(&buf_done[b], 8);
        }
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.x);
        prefetch_tmap(&maps.w);
        if (a.gated) prefetch_tmap(&maps.v);
        if (by_tma) prefetch_tmap(&maps.out);
        if (res_tma) prefetch_tmap(&maps.res);
    }
    if (warp == 1) tmem_alloc_pair(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either is signalled from the other
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    pdl_trigger();
    auto give_up = [&]() {
        abort_flag = 1;
        status_or(a.status, MOE_DEV_TIMEOUT);
    };
    auto first = [&](const ManySched::Place& i, int& r0, int& f0) {  // this CTA's first row, the first feature of tile i
        int tt, tn;
        sched.tiles(i, tt, tn);
        r0 = tt * 256 + rank * 128;
        f0 = tn * per_tile;
    };
    if (warp == 0) {  // roles of elected lanes as in the other kernel
        if (elect_one()) {  // TMA producer of this CTA's halves
            const CUtensorMap* wmap = a.gated && rank == 1 ? &maps.v : &maps.w;
            int it = 0;
            RingPos at;
            for (auto i = sched.begin(pair); i.tile < sched.total && !abort_flag; sched.next(i, pairs)) {
                int t0, n0;
                first(i, t0, n0);
                if (!a.gated) n0 += rank * half;
                for (int k = 0; k < a.nk; k += 2, ++it, at.next(kManyStages)) {
                    const int s = at.slot, parts = min(2, a.nk - k);
                    if (!mbar_wait_suspended(&empty[s], at.parity ^ 1)) {
                        give_up();
                        break;
                    }
                    const uint32_t base = smem_u32(smem + s * kManyStageBytes);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * parts * (kLinA + half * 128));
                    const uint32_t bar = map_rank(smem_u32(&full[s]), 0);
                    for (int h = 0; h < parts; ++h) {
                        tma_load_pair(base + h * kManyHalf, &maps.x, (k + h) * kLinK, t0, bar);
                        tma_load_pair(base + h * kManyHalf + kLinA, wmap, (k + h) * kLinK, n0, bar);
                    }
                }
            }
            if (rank == 0)  // whoever gives up, none of the pair's copies is in flight when its CTAs end
                for (int i = it < kManyStages ? it : kManyStages; i > 0; --i) {
                    at.back(kManyStages);
                    mbar_wait_suspended(&full[at.slot], at.parity);
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {  // MMA issuer of the pair
            const uint32_t idesc = idesc_f16kind(256, a.width, a.f16);
            int n = 0;
            RingPos ring;
            for (int64_t i = pair; i < sched.total && !abort_flag; i += pairs, ++n) {
                const int b = n & 1;
                if (!mbar_wait_suspended(&acc_empty[b], ((n >> 1) & 1) ^ 1)) {
                    give_up();
                    break;
                }
                tc_fence_after();
                for (int k = 0; k < a.nk; k += 2, ring.next(kManyStages)) {
                    const int s = ring.slot, parts = min(2, a.nk - k);
                    if (!mbar_wait_suspended(&full[s], ring.parity)) {
                        give_up();
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc(smem_u32(smem + s * kManyStageBytes), 16, 1024, kLayoutSw128);
                    for (int h = 0; h < parts; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {  // K 16 per MMA: 32 bytes (two units) along the swizzled row
                            const uint64_t at = ad + h * (kManyHalf >> 4) + 2 * j;
                            mma_f16kind<1>(tmem + 256 * b, at, at + (kLinA >> 4), idesc, (k | h | j) != 0);
                        }
                    tc_commit_pair(&empty[s], 3);
                }
                tc_commit_pair(&acc_full[b], 3);
            }
        }
        __syncwarp();
    } else if (warp >= 2 && warp < 10) {
        const int q = warp & 3, side = (warp - 2) >> 2;  // lane quarter, parity of the columns' 16s
        const int row = 32 * q + lane, sw = (row >> 1) & 3;
        int n = 0;
        uint32_t pass = 0;
        for (int64_t i = pair; i < sched.total && !abort_flag; i += pairs, ++n) {
            const int b = n & 1;
            if (!__all_sync(0xffffffffu, mbar_wait_suspended(&acc_full[b], (n >> 1) & 1))) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t trow = tmem + 256 * b + ((uint32_t)(32 * q) << 16);
            for (int p = 0; p < passes; ++p, ++pass) {
                const int buf = pass & 1;
                if (!__all_sync(0xffffffffu, mbar_wait_suspended(&buf_ready[buf], (pass >> 1) & 1)))
                    give_up();  // carries on: the row movers stop, and with them this loop
                for (int c = 4 * p + side; c < min(4 * p + 4, 2 * subs); c += 2) {  // 16 features each
                    float z[16], u[16];
                    tmem_ld_16(trow + 16 * c, reinterpret_cast<uint32_t(&)[16]>(z));
                    if (a.gated) tmem_ld_16(trow + half + 16 * c, reinterpret_cast<uint32_t(&)[16]>(u));
                    tmem_ld_wait();
                    uint8_t* line = rows_s + buf * 2 * kManySub + ((c >> 1) & 1) * kManySub + row * 64;
                    uint4* p0 = reinterpret_cast<uint4*>(line + (((2 * (c & 1)) ^ sw) << 4));
                    uint4* p1 = reinterpret_cast<uint4*>(line + (((2 * (c & 1) + 1) ^ sw) << 4));
                    uint32_t rw[8] = {};
                    if (a.res) {
                        *reinterpret_cast<uint4*>(rw) = *p0;
                        *reinterpret_cast<uint4*>(rw + 4) = *p1;
                    }
                    uint32_t ow[8];
                    const float* bias = bias_s[buf] + 16 * (c & 3);
                    combine16(a, bias, bias + 64, z, u, rw, ow);
                    *p0 = *reinterpret_cast<uint4*>(ow);
                    *p1 = *reinterpret_cast<uint4*>(ow + 4);
                    __syncwarp();
                }
                if (by_tma) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&buf_done[buf]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(map_rank(smem_u32(&acc_empty[b]), 0));
        }
    } else if (warp >= 10 && (warp == 10 || !by_tma)) {  // row movers
        struct {
            ManySched::Place at;
            int p;             // pass of the tile
            uint32_t pass;     // of all this CTA's
        } next_in{sched.begin(pair), 0, 0}, out_of = next_in;  // the pass to make a buffer ready for, and to move out
        const auto go_on = [&](auto& to) {
            ++to.pass;
            if (++to.p == passes) {
                to.p = 0;
                sched.next(to.at, pairs);
            }
        };
        const int first_row = 32 * (warp - 10);  // of this warp's share, without TMA
        // row r, feature f < 64 of a buffer
        const auto element = [&](int buf, int r, int f) {
            uint8_t* line = rows_s + (2 * buf + (f >> 5)) * kManySub + r * 64;
            return reinterpret_cast<uint16_t*>(line + ((((f & 31) >> 3) ^ ((r >> 1) & 3)) << 4) + (f & 7) * 2);
        };
        // whether an element stands at an odd multiple of 2 bytes
        const auto odd_at = [](const uint16_t* at) { return (int)((reinterpret_cast<uintptr_t>(at) >> 1) & 1); };
        // f with the oddness of the even and of the odd rows from one that starts `odd`, known when compiled
        const auto with_parity = [](int odd, int64_t ld, auto&& f) {
            using Is = std::integral_constant<int, 1>;
            using Not = std::integral_constant<int, 0>;
            if (ld & 1) {
                if (odd) f(Is{}, Not{});
                else f(Not{}, Is{});
            } else {
                if (odd) f(Is{}, Is{});
                else f(Not{}, Not{});
            }
        };
        // makes a buffer ready for the next pass, if there is one: its biases, and the residual if there is one
        const auto prepare = [&]() {
            if (next_in.at.tile >= sched.total) return;
            const int buf = (int)(next_in.pass & 1);
            int r0, f0;
            first(next_in.at, r0, f0);
            const int p = next_in.p, fp = f0 + 64 * p, pieces = min(2, subs - 2 * p);
            if ((a.bias || a.bias_mul) && warp == 10) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float* src = j < 2 ? a.bias : a.bias_mul;
                    const int f = fp + lane + 32 * (j & 1);
                    bias_s[buf][lane + 32 * j] = src && f < a.N ? __ldg(src + f) : 0.f;
                }
            }
            if (a.res && !by_tma) {
                const uint16_t* src = static_cast<const uint16_t*>(a.res) + ((int64_t)r0 + first_row) * a.ldr + fp;
                const int rows = min(32, a.T - r0 - first_row), in = min(32 * pieces, a.N - fp);
                const int odd_lane = odd_at(src + lane * a.ldr);
                // the single features at the ends, a row a lane; then two features a lane of every row: all in flight
                const bool head = odd_lane && in > 0 && lane < rows, tail = ((in - odd_lane) & 1) && in > odd_lane && lane < rows;
                const uint16_t h0 = head ? __ldcg(src + lane * a.ldr) : (uint16_t)0;
                const uint16_t h1 = tail ? __ldcg(src + lane * a.ldr + in - 1) : (uint16_t)0;
                with_parity(odd_at(src), a.ldr, [&](auto even_rows, auto odd_rows) {
                    constexpr int O[2] = {even_rows.value, odd_rows.value};
                    const bool pair[2] = {2 * lane + 1 < in, 2 * lane + 2 < in};
                    uint32_t v[32];
#pragma unroll
                    for (int r = 0; r < 32; ++r) {
                        const int odd = O[r & 1];
                        v[r] = r < rows && pair[odd]
                                   ? __ldcg(reinterpret_cast<const uint32_t*>(src + r * a.ldr + 2 * lane + odd)) : 0u;
                    }
#pragma unroll
                    for (int r = 0; r < 32; ++r) {
                        const int odd = O[r & 1], f = 2 * lane + odd;
                        if (!odd) {
                            if (pair[0]) *reinterpret_cast<uint32_t*>(element(buf, first_row + r, f)) = v[r];
                        } else if (pair[1]) {
                            *element(buf, first_row + r, f) = (uint16_t)v[r];
                            *element(buf, first_row + r, f + 1) = (uint16_t)(v[r] >> 16);
                        }
                    }
                });
                if (head) *element(buf, first_row + lane, 0) = h0;
                if (tail) *element(buf, first_row + lane, in - 1) = h1;
            }
            __syncwarp();
            if (lane == 0) {
                if (!res_tma) {
                    mbar_arrive(&buf_ready[buf]);
                } else {
                    mbar_arrive_expect_tx(&buf_ready[buf], pieces * kManySub);
                    for (int s = 0; s < pieces; ++s)
                        tma_load_2d(rows_s + (2 * buf + s) * kManySub, &maps.res, fp + 32 * s, r0, &buf_ready[buf]);
                }
            }
            __syncwarp();
            go_on(next_in);
        };
        prepare();
        prepare();
        bool gave_up = false;
        for (; out_of.at.tile < sched.total; go_on(out_of)) {
            const int buf = (int)(out_of.pass & 1);
            if (!__all_sync(0xffffffffu, mbar_wait_suspended(&buf_done[buf], (out_of.pass >> 1) & 1)) ||
                __any_sync(0xffffffffu, abort_flag)) {
                give_up();
                gave_up = true;
                break;
            }
            int r0, f0;
            first(out_of.at, r0, f0);
            const int p = out_of.p, fp = f0 + 64 * p, pieces = min(2, subs - 2 * p);
            if (!by_tma) {
                uint16_t* dst = static_cast<uint16_t*>(a.out) + ((int64_t)r0 + first_row) * a.ldo + fp;
                const int rows = min(32, a.T - r0 - first_row), in = min(32 * pieces, a.N - fp);
                const int odd_lane = odd_at(dst + lane * a.ldo);
                if (lane < rows) {
                    if (odd_lane && in > 0) dst[lane * a.ldo] = *element(buf, first_row + lane, 0);
                    if (((in - odd_lane) & 1) && in > odd_lane)
                        dst[lane * a.ldo + in - 1] = *element(buf, first_row + lane, in - 1);
                }
                with_parity(odd_at(dst), a.ldo, [&](auto even_rows, auto odd_rows) {
                    constexpr int O[2] = {even_rows.value, odd_rows.value};
                    const bool pair[2] = {2 * lane + 1 < in, 2 * lane + 2 < in};
#pragma unroll
                    for (int b = 0; b < 32; b += 8) {
                        uint32_t v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int r = first_row + b + i, odd = O[i & 1], f = 2 * lane + odd;
                            if (!odd) v[i] = *reinterpret_cast<const uint32_t*>(element(buf, r, f));
                            else v[i] = *element(buf, r, f) | (uint32_t)*element(buf, r, min(f + 1, 63)) << 16;
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int odd = O[i & 1];
                            if (b + i < rows && pair[odd])
                                *reinterpret_cast<uint32_t*>(dst + (b + i) * a.ldo + 2 * lane + odd) = v[i];
                        }
                    }
                });
            } else if (lane == 0) {
                for (int s = 0; s < pieces; ++s)
                    if (fp + 32 * s < a.N && r0 < a.T)
                        tma_store_2d(&maps.out, rows_s + (2 * buf + s) * kManySub, fp + 32 * s, r0);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            __syncwarp();
            prepare();
        }
        if (gave_up)  // wait (bounded) for the residual copies in flight
            for (uint32_t j = out_of.pass; j != next_in.pass; ++j) mbar_wait_suspended(&buf_ready[j & 1], (j >> 1) & 1);
        if (lane == 0 && by_tma) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    cluster_sync();  // the peer's copies, MMAs and arrivals into this CTA are done
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---- host ------------------------------------------------------------------------------------------
template <typename K>
cudaError_t launch_clusters(K* kernel, int smem_max, std::atomic<uint64_t>& allowed, dim3 grid, int cluster,
                            int threads, int smem, const LinMaps& m, const LinArgs& a, cudaStream_t st) {
    const cudaError_t err = allow_large_launch(kernel, smem_max, allowed);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, m, a);
}

template <bool PAIR>
cudaError_t launch_few(const LinMaps& m, const LinArgs& a, int splits, int N, cudaStream_t st) {
    using F = Few<PAIR>;
    const int per_tile = F::kW * F::kCtas / (a.gated ? 2 : 1), cluster = splits * F::kCtas;
    const dim3 grid((N + per_tile - 1) / per_tile * cluster, (a.T + a.rows_t - 1) / a.rows_t);
    static std::atomic<uint64_t> allowed{0};
    return launch_clusters(linear_few_kernel<PAIR>, kCtaSmemMax, allowed, grid, cluster, kFewThreads,
                           F::smem(a.rows_t, splits, a.stages), m, a, st);
}

}  // namespace

cudaError_t launch_linear(const moe_linear_desc& d, const void* x, const void* w, const void* w_mul,
                          const float* bias, const float* bias_mul, const void* residual, void* out,
                          int32_t* status, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    LinArgs a{};
    a.T = d.T; a.N = d.N; a.nk = (d.K + kLinK - 1) / kLinK;
    a.func = d.func; a.gated = w_mul != nullptr; a.f16 = d.dtype == MOE_DT_F16;
    a.ldr = d.ldr; a.ldo = d.ldo;
    a.bias = bias; a.bias_mul = bias_mul; a.res = residual; a.out = out; a.status = status;
    const LinPlan plan = plan_linear(d.T, d.N, a.nk, a.gated, sms);
    LinMaps m{};
    // rows of W per box, and rows of x
    const int box_w = plan.few ? (plan.pair ? 64 : 128) / (a.gated ? 2 : 1) : plan.width / 2;
    const int box_x = !plan.few ? 128 : plan.pair ? plan.rows_t / 2 : plan.rows_t;
    if (!encode_rows16(&m.x, x, d.K, d.T, d.ldx, box_x, kLinK) || !encode_rows16(&m.w, w, d.K, d.N, d.ldw, box_w, kLinK) ||
        (a.gated && !encode_rows16(&m.v, w_mul, d.K, d.N, d.ldw, box_w, kLinK)))
        return cudaErrorInvalidValue;
    if (plan.few) {
        a.rows_t = plan.rows_t;
        a.stages = plan.stages;
        return plan.pair ? launch_few<true>(m, a, plan.splits, d.N, st) : launch_few<false>(m, a, plan.splits, d.N, st);
    }
    // TMA addresses rows that start at multiples of 16 bytes, and writes whole ones: where a row ends inside 16 bytes, what lies
    // behind it is written too
    a.width = plan.width;
    a.tma_rows = d.N % 8 == 0 && rows_aligned(out, d.ldo, 16) && (!residual || rows_aligned(residual, d.ldr, 16));
    if (a.tma_rows && (!encode_rows16(&m.out, out, d.N, d.T, d.ldo, 128, 32) ||
                       (residual && !encode_rows16(&m.res, residual, d.N, d.T, d.ldr, 128, 32))))
        return cudaErrorInvalidValue;
    const int64_t total = ManySched(d.T, d.N, a.gated ? a.width / 2 : a.width).total;
    const int pairs = (int)(total < sms / 2 ? total : sms / 2);
    static std::atomic<uint64_t> allowed{0};
    return launch_clusters(linear_many_kernel, kManySmem, allowed, dim3(2 * pairs), 2, kManyThreads, kManySmem, m, a, st);
}

}  // namespace moe
