// linear.cu -- y = f(x W^T + b) [* (x V^T + c)] [+ r], fp32 sums, one rounding.
//
// Two kernels on tcgen05.mma.kind::f16, both fed by TMA (64 elements of K per stage, 128-byte
// swizzled rows; what lies beyond a matrix reads as zero) into accumulators in tensor memory:
//
//   linear_few_kernel   few rows.  The time is that of streaming the weights, so the weights are
//       the MMA's 128-row operand and the rows of x its N side (16 to 256 columns): each weight
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
#include <cudaTypedefs.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

using namespace tc;

constexpr uint64_t kLinWaitLimit = 1ull << 26;  // polls before a wait is declared stuck
constexpr int kLinK = 64;                       // K elements per stage (128 bytes per row)
constexpr int kLinA = 128 * 128;                // bytes of a 128-row operand stage

struct LinMaps {
    CUtensorMap x, w, v, res, out;
};

struct LinArgs {
    int T, N, nk;       // nk: stages of K in all
    int func, gated, f16;
    int rows_t, stages; // few rows: rows of x per tile, stages of the ring
    int tma_rows;       // many rows: out and the residual go by TMA
    int wave;           // many rows: CTA pairs the device holds
    int64_t ldr, ldo;
    const float *bias, *bias_mul;
    const void* res;
    void* out;
    int32_t* status;
};

// ---- cluster and CTA-pair primitives -----------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared-memory location `saddr` in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void arrive_cluster(uint32_t mapped_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapped_bar) : "memory");
}
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
// Arrive on `bar` of both CTAs of the pair once this thread's earlier MMAs have completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)), "h"((uint16_t)3) : "memory");
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
__device__ __forceinline__ float apply_func(int func, float z) {
    switch (func) {
        case MOE_FUNC_SILU: return __fdividef(z, 1.f + __expf(-z));
        case MOE_FUNC_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678f));
        // 0.5 (1 + tanh u) = sigmoid(2 u)
        case MOE_FUNC_GELU_TANH: return z / (1.f + __expf(-1.5957691f * (z + 0.044715f * z * z * z)));
        case MOE_FUNC_RELU: return fmaxf(z, 0.f);
    }
    return z;
}
__device__ __forceinline__ float unpack16(uint32_t h, bool f16) {
    return f16 ? __half2float(__ushort_as_half((unsigned short)h)) : __uint_as_float(h << 16);
}
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi, bool f16) {
    uint32_t r;
    if (f16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// C consecutive outputs of row t from feature n on: bias, function, factor, residual, one rounding.
// u: the factor's sums (gated).  vec: every row starts at a multiple of 2 C bytes.
template <int C>
__device__ __forceinline__ void finish(const LinArgs& a, int64_t t, int n, float (&z)[C], const float (&u)[C],
                                       bool vec) {
    const bool f16 = a.f16;
    uint16_t* out = static_cast<uint16_t*>(a.out) + t * a.ldo + n;
    const uint16_t* res = a.res ? static_cast<const uint16_t*>(a.res) + t * a.ldr + n : nullptr;
    const bool full = vec && n + C <= a.N;
    uint32_t rw[C / 2];
    if (res && full) {
#pragma unroll
        for (int i = 0; i < C / 2; i += C >= 8 ? 4 : 2) {
            if constexpr (C >= 8) {
                const uint4 q = *reinterpret_cast<const uint4*>(res + 2 * i);
                rw[i] = q.x; rw[i + 1] = q.y; rw[i + 2] = q.z; rw[i + 3] = q.w;
            } else {
                const uint2 q = *reinterpret_cast<const uint2*>(res + 2 * i);
                rw[i] = q.x; rw[i + 1] = q.y;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const bool in = n + i < a.N;
        if (a.bias && in) z[i] += __ldg(a.bias + n + i);
        z[i] = apply_func(a.func, z[i]);
        if (a.gated) z[i] *= u[i] + (a.bias_mul && in ? __ldg(a.bias_mul + n + i) : 0.f);
        if (res) {
            if (full) z[i] += unpack16(i & 1 ? rw[i / 2] >> 16 : rw[i / 2] & 0xFFFFu, f16);
            else if (in) z[i] += unpack16(res[i], f16);
        }
    }
    uint32_t ow[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) ow[i] = pack16x2(z[2 * i], z[2 * i + 1], f16);
    if (full) {
#pragma unroll
        for (int i = 0; i < C / 2; i += C >= 8 ? 4 : 2) {
            if constexpr (C >= 8)
                *reinterpret_cast<uint4*>(out + 2 * i) = make_uint4(ow[i], ow[i + 1], ow[i + 2], ow[i + 3]);
            else
                *reinterpret_cast<uint2*>(out + 2 * i) = make_uint2(ow[i], ow[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (n + i < a.N) out[i] = (uint16_t)(i & 1 ? ow[i / 2] >> 16 : ow[i / 2] & 0xFFFFu);
    }
}

// 16 outputs of one row, biases in shared memory, the residual's 16 values packed in rw (zeros
// without one), to packed results.
__device__ __forceinline__ void combine16(const LinArgs& a, const float* bias, const float* bias_mul,
                                          float (&z)[16], const float (&u)[16], const uint32_t (&rw)[8],
                                          uint32_t (&ow)[8]) {
    const bool f16 = a.f16;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 b = a.bias ? *reinterpret_cast<const float4*>(bias + i) : make_float4(0, 0, 0, 0);
        const float4 c = a.bias_mul ? *reinterpret_cast<const float4*>(bias_mul + i) : make_float4(0, 0, 0, 0);
        const float bb[4] = {b.x, b.y, b.z, b.w}, cc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float y = apply_func(a.func, z[i + j] + bb[j]);
            if (a.gated) y *= u[i + j] + cc[j];
            if (a.res) y += unpack16(j & 1 ? rw[(i + j) / 2] >> 16 : rw[(i + j) / 2] & 0xFFFFu, f16);
            z[i + j] = y;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ow[i] = pack16x2(z[2 * i], z[2 * i + 1], f16);
}

// Whether rows of `p` (ld elements apart) all start at multiples of `bytes`.
__host__ __device__ __forceinline__ bool rows_aligned(const void* p, int64_t ld, int bytes) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(2 * ld)) & (uintptr_t)(bytes - 1)) == 0;
}

// ------------------------------------------------------------------------------------------
// Few rows.  grid (tiles of W rows * splits of K, tiles of x rows), clusters of `splits` CTAs.  A tile
// is 128 rows of W, or 64 of W and 64 of V.  Warp 0 loads, warp 1 issues the MMAs, warps 2-5 move
// the accumulator (lane = W row, column = row of x) to shared memory, then all six warps add
// the cluster's partial sums: CTA r takes columns r, r + splits, ...
// ------------------------------------------------------------------------------------------
constexpr int kFewThreads = 192;

__global__ void __launch_bounds__(kFewThreads)
linear_few_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinArgs a) {
    extern __shared__ uint8_t lin_smem[];
    __shared__ uint64_t full[8], empty[8], acc_full;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_smem) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t splits;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(splits));
    const uint32_t rank = cluster_rank();
    const int per_tile = a.gated ? 64 : 128;
    const int n0 = (int)(blockIdx.x / splits) * per_tile;
    const int t0 = (int)blockIdx.y * a.rows_t;
    const int NT = a.rows_t;
    const int k_begin = (int)((int64_t)a.nk * rank / splits), k_end = (int)((int64_t)a.nk * (rank + 1) / splits);
    const int stage_bytes = kLinA + NT * 128;
    uint32_t tm_cols = 32;
    while (tm_cols < (uint32_t)NT) tm_cols *= 2;
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.x);
        prefetch_tmap(&maps.w);
        if (a.gated) prefetch_tmap(&maps.v);
    }
    if (warp == 1) tmem_alloc(&tmem_slot, tm_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();
    pdl_trigger();  // after the allocation, so that a waiting successor cannot hold the columns
    auto give_up = [&]() {
        abort_flag = 1;
        status_or(a.status, MOE_DEV_TIMEOUT);
    };
    const int steps = k_end - k_begin;
    if (warp == 0 && lane == 0) {
        int issued = 0;
        for (int i = 0; i < steps && !abort_flag; ++i) {
            const int s = i % a.stages;
            if (!mbar_wait_bounded(&empty[s], ((i / a.stages) & 1) ^ 1, kLinWaitLimit)) {
                give_up();
                break;
            }
            uint8_t* base = smem + s * stage_bytes;
            const int kx = (k_begin + i) * kLinK;
            mbar_arrive_expect_tx(&full[s], stage_bytes);
            tma_load_2d(base, &maps.w, kx, n0, &full[s]);
            if (a.gated) tma_load_2d(base + kLinA / 2, &maps.v, kx, n0, &full[s]);
            tma_load_2d(base + kLinA, &maps.x, kx, t0, &full[s]);
            ++issued;
        }
        if (abort_flag)  // wait (bounded) for the copies still in flight
            for (int i = issued - 1; i >= 0 && i >= issued - a.stages; --i)
                mbar_wait_bounded(&full[i % a.stages], (i / a.stages) & 1, kLinWaitLimit);
    } else if (warp == 1 && lane == 0) {
        const uint32_t idesc = idesc_f16kind(128, NT, a.f16);
        int i = 0;
        for (; i < steps; ++i) {
            const int s = i % a.stages;
            if (!mbar_wait_bounded(&full[s], (i / a.stages) & 1, kLinWaitLimit) || abort_flag) {
                give_up();
                break;
            }
            tc_fence_after();
            const uint32_t sb = smem_u32(smem + s * stage_bytes);
#pragma unroll
            for (int j = 0; j < 4; ++j)  // K 16 per MMA: 32 bytes along the swizzled row
                mma_f16kind<0>(tmem, smem_desc(sb + 32 * j, 16, 1024, kLayoutSw128),
                               smem_desc(sb + kLinA + 32 * j, 16, 1024, kLayoutSw128), idesc, (i | j) != 0);
            tc_commit(&empty[s]);
        }
        tc_commit(&acc_full);  // arrives when every MMA has completed
        mbar_wait_bounded(&acc_full, 0, kLinWaitLimit);
    }
    const int ncols = min(NT, a.T - t0);
    float* part = reinterpret_cast<float*>(smem);  // [column][128]; the ring is idle by then
    if (warp >= 2) {
        if (!mbar_wait_bounded(&acc_full, 0, kLinWaitLimit)) give_up();
        tc_fence_after();
        const int q = warp & 3;
        for (int c = 0; c < ncols; c += 16) {
            uint32_t v[16];
            tmem_ld_16(tmem + ((uint32_t)(32 * q) << 16) + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < NT) part[(c + i) * 128 + 32 * q + lane] = __uint_as_float(v[i]);
        }
        tc_fence_before();
    }
    __syncthreads();
    cluster_sync();  // every partial sum is in shared memory
    {
        const bool vec = rows_aligned(a.out, a.ldo, 8) && (!a.res || rows_aligned(a.res, a.ldr, 8));
        const uint32_t pbase = smem_u32(part);
        for (int c = (int)rank + (int)splits * warp; c < ncols; c += (int)splits * (kFewThreads / 32)) {
            float z[4] = {0.f, 0.f, 0.f, 0.f}, u[4];
            for (uint32_t s = 0; s < splits; ++s) {
                const float4 p = ld_cluster_f4(map_rank(pbase + (uint32_t)(c * 128 + 4 * lane) * 4, s));
                z[0] += p.x; z[1] += p.y; z[2] += p.z; z[3] += p.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = __shfl_down_sync(0xffffffffu, z[i], 16);
            const int n = n0 + 4 * lane;
            if (n < a.N && (!a.gated || lane < 16)) finish<4>(a, (int64_t)t0 + c, n, z, u, vec);
        }
    }
    cluster_sync();  // no CTA leaves while others read its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, tm_cols);
    }
}

// ------------------------------------------------------------------------------------------
// Many rows.  Clusters of two CTAs, one per SM; pair p takes tiles p, p + pairs, ...  A tile is 256 rows
// of x by 256 rows of W (gated: 128 of W and 128 of V); each CTA holds 128 rows of x and all columns.
// Tiles of a last wave that would leave half of the pairs idle are cut in two by columns.  Warp 0
// loads, warp 1 of the leading CTA issues the MMAs, warps 2-9 (two per lane quarter, half the
// columns each) turn accumulators into rows.  Rows go out, and the residual comes in, by TMA through
// a 64 KB staging area (128-byte swizzled, so a thread per row meets no bank conflicts): the next
// tile's residual loads while its MMAs run.  Rows that TMA cannot address (not 16-byte aligned) are
// read and written by the threads.
// ------------------------------------------------------------------------------------------
constexpr int kManyThreads = 320;
constexpr int kManyStages = 5;
constexpr int kManyStageBytes = 2 * kLinA;  // 128 rows of x, at most 128 of W
constexpr int kManyBox = 64 * 128;          // bytes of a 64-row box of weights
constexpr int kManySmem = kManyStages * kManyStageBytes + 4 * kLinA + 1024;
constexpr int kManyGroup = 8;  // row tiles that share a pass over the weights

struct ManyTile {
    int t0, f0, boxes;  // first row, first feature, 64-row weight boxes per CTA (2, or 1: half a tile)
};

struct ManySched {
    int tiles_t, tiles_n, gated;
    int64_t whole, total;
    __host__ __device__ ManySched(int T, int N, int gated_, int pairs) : gated(gated_) {
        tiles_t = (int)(((int64_t)T + 255) / 256);
        tiles_n = (N + (gated ? 127 : 255)) / (gated ? 128 : 256);
        const int64_t all = (int64_t)tiles_t * tiles_n, last = all % pairs;
        const int64_t cut = 2 * last <= pairs ? last : 0;
        whole = all - cut;
        total = whole + 2 * cut;
    }
    __device__ __forceinline__ ManyTile tile(int64_t i) const {
        const bool half = i >= whole;
        const int64_t w = half ? whole + (i - whole) / 2 : i;
        const int64_t per = (int64_t)kManyGroup * tiles_n;
        const int g = (int)(w / per), rest = (int)(w % per);
        const int rows = min(kManyGroup, tiles_t - g * kManyGroup);
        ManyTile r;
        r.t0 = (g * kManyGroup + rest % rows) * 256;
        r.boxes = half ? 1 : 2;
        r.f0 = (rest / rows) * (gated ? 128 : 256) + (half ? (int)((i - whole) & 1) * (gated ? 64 : 128) : 0);
        return r;
    }
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(smem_u32(src)) : "memory");
}
__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__global__ void __launch_bounds__(kManyThreads, 1)
linear_many_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinArgs a) {
    extern __shared__ uint8_t lin_smem[];
    __shared__ uint64_t full[kManyStages], empty[kManyStages], acc_full[2], acc_empty[2], res_full;
    __shared__ __align__(16) float bias_s[256];  // gated: 128 of bias, 128 of bias_mul
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag, stop;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_smem) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = smem + kManyStages * kManyStageBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const ManySched sched(a.T, a.N, a.gated, a.wave);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kManyStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 16);  // the epilogue warps of both CTAs
        }
        mbar_init(&res_full, 1);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&maps.x);
        prefetch_tmap(&maps.w);
        if (a.gated) prefetch_tmap(&maps.v);
        if (a.tma_rows) prefetch_tmap(&maps.out);
        if (a.tma_rows && a.res) prefetch_tmap(&maps.res);
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
    if (warp == 0 && lane == 0) {  // TMA producer of this CTA's halves
        const CUtensorMap* wmap = a.gated && rank == 1 ? &maps.v : &maps.w;
        int it = 0;
        for (int64_t i = pair; i < sched.total && !abort_flag; i += pairs) {
            const ManyTile tl = sched.tile(i);
            const int t0 = tl.t0 + (int)rank * 128;
            const int n0 = tl.f0 + (a.gated ? 0 : (int)rank * 64 * tl.boxes);
            for (int k = 0; k < a.nk; ++k, ++it) {
                const int s = it % kManyStages;
                if (!mbar_wait_bounded(&empty[s], ((it / kManyStages) & 1) ^ 1, kLinWaitLimit) || abort_flag) {
                    give_up();
                    break;
                }
                const uint32_t base = smem_u32(smem + s * kManyStageBytes);
                if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (kLinA + tl.boxes * kManyBox));
                const uint32_t bar = map_rank(smem_u32(&full[s]), 0);
                tma_load_pair(base, &maps.x, k * kLinK, t0, bar);
                tma_load_pair(base + kLinA, wmap, k * kLinK, n0, bar);
                if (tl.boxes == 2) tma_load_pair(base + kLinA + kManyBox, wmap, k * kLinK, n0 + 64, bar);
            }
        }
        if (abort_flag && rank == 0)  // wait (bounded) for the pair's copies still in flight
            for (int j = it - 1; j >= 0 && j >= it - kManyStages; --j)
                mbar_wait_bounded(&full[j % kManyStages], (j / kManyStages) & 1, kLinWaitLimit);
    } else if (warp == 1 && lane == 0 && rank == 0) {  // MMA issuer of the pair
        int it = 0, n = 0;
        for (int64_t i = pair; i < sched.total && !abort_flag; i += pairs, ++n) {
            const uint32_t idesc = idesc_f16kind(256, 128 * sched.tile(i).boxes, a.f16);
            const int b = n & 1;
            if (!mbar_wait_bounded(&acc_empty[b], ((n >> 1) & 1) ^ 1, kLinWaitLimit)) {
                give_up();
                break;
            }
            tc_fence_after();
            for (int k = 0; k < a.nk; ++k, ++it) {
                const int s = it % kManyStages;
                if (!mbar_wait_bounded(&full[s], (it / kManyStages) & 1, kLinWaitLimit) || abort_flag) {
                    give_up();
                    break;
                }
                tc_fence_after();
                const uint32_t sb = smem_u32(smem + s * kManyStageBytes);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_f16kind<1>(tmem + 256 * b, smem_desc(sb + 32 * j, 16, 1024, kLayoutSw128),
                                   smem_desc(sb + kLinA + 32 * j, 16, 1024, kLayoutSw128), idesc, (k | j) != 0);
                tc_commit_pair(&empty[s]);
            }
            tc_commit_pair(&acc_full[b]);
        }
    } else if (warp >= 2) {
        const int q = warp & 3, side = (warp - 2) >> 2;  // lane quarter, half of the columns
        const int etid = threadIdx.x - 64;
        const int row = 32 * q + lane;
        const bool leader = etid == 0;
        const bool by_tma = a.tma_rows, res_tma = by_tma && a.res;
        const bool vec = rows_aligned(a.out, a.ldo, 16) && (!a.res || rows_aligned(a.res, a.ldr, 16));
        auto load_residual = [&](int64_t i) {  // a tile's residual rows into the staging area
            const ManyTile tl = sched.tile(i);
            const int subs = (a.gated ? 1 : 2) * tl.boxes;
            mbar_arrive_expect_tx(&res_full, subs * kLinA);
            for (int s = 0; s < subs; ++s)
                tma_load_2d(staging + s * kLinA, &maps.res, tl.f0 + 64 * s, tl.t0 + (int)rank * 128, &res_full);
        };
        if (leader && res_tma && pair < sched.total) load_residual(pair);
        int n = 0;
        bool ok = true;
        for (int64_t i = pair; i < sched.total; i += pairs, ++n) {
            const int b = n & 1;
            const ManyTile tl = sched.tile(i);
            const int subs = (a.gated ? 1 : 2) * tl.boxes;  // 64-feature pieces of the tile
            if (a.bias || a.bias_mul) {
                const bool second = a.gated && etid >= 128;
                const float* src = second ? a.bias_mul : a.bias;
                const int f = tl.f0 + (second ? etid - 128 : etid);
                bias_s[etid] = src && f < a.N ? __ldg(src + f) : 0.f;
            }
            ok = mbar_wait_bounded(&acc_full[b], (n >> 1) & 1, kLinWaitLimit) && ok;
            if (res_tma) ok = mbar_wait_bounded(&res_full, n & 1, kLinWaitLimit) && ok;
            if (!ok) give_up();
            epilogue_barrier();  // bias_s is written; the staging area is free or holds the residual
            tc_fence_after();
            const uint32_t trow = tmem + 256 * b + ((uint32_t)(32 * q) << 16);
            const int64_t t = (int64_t)tl.t0 + rank * 128 + row;
            for (int c = side; c < subs * 4; c += 2) {  // 16 features each
                float z[16], u[16];
                tmem_ld_16(trow + 16 * c, reinterpret_cast<uint32_t(&)[16]>(z));
                if (a.gated) tmem_ld_16(trow + 64 * tl.boxes + 16 * c, reinterpret_cast<uint32_t(&)[16]>(u));
                tmem_ld_wait();
                if (by_tma) {
                    uint8_t* line = staging + (c >> 2) * kLinA + row * 128;
                    uint4* p0 = reinterpret_cast<uint4*>(line + (((2 * (c & 3)) ^ (row & 7)) << 4));
                    uint4* p1 = reinterpret_cast<uint4*>(line + (((2 * (c & 3) + 1) ^ (row & 7)) << 4));
                    uint32_t rw[8] = {};
                    if (res_tma) {
                        *reinterpret_cast<uint4*>(rw) = *p0;
                        *reinterpret_cast<uint4*>(rw + 4) = *p1;
                    }
                    uint32_t ow[8];
                    combine16(a, bias_s + 16 * c, bias_s + 128 + 16 * c, z, u, rw, ow);
                    *p0 = *reinterpret_cast<uint4*>(ow);
                    *p1 = *reinterpret_cast<uint4*>(ow + 4);
                } else if (t < a.T && tl.f0 + 16 * c < a.N) {
                    finish<16>(a, t, tl.f0 + 16 * c, z, u, vec);
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(map_rank(smem_u32(&acc_empty[b]), 0));
            if (by_tma) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (leader) stop = abort_flag;  // one answer for all the epilogue's warps
            epilogue_barrier();
            if (leader && by_tma) {
                for (int s = 0; s < subs; ++s)
                    if (tl.f0 + 64 * s < a.N && tl.t0 + (int)rank * 128 < a.T)
                        tma_store_2d(&maps.out, staging + s * kLinA, tl.f0 + 64 * s, tl.t0 + (int)rank * 128);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                if (res_tma && i + pairs < sched.total && !stop) load_residual(i + pairs);
            }
            if (stop) break;
        }
        if (leader && by_tma) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    cluster_sync();  // the peer's copies, MMAs and arrivals into this CTA are done
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---- host ------------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// [rows][cols] 16-bit elements, rows ld apart; boxes of 64 columns x box_rows, 128-byte swizzle.
bool encode16(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
    const auto fn = encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    cuuint32_t box[2] = {(cuuint32_t)kLinK, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t launch_clusters(K* kernel, dim3 grid, int cluster, int threads, int smem, const LinMaps& m,
                            const LinArgs& a, cudaStream_t st) {
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
    LinMaps m{};
    if (d.T <= 512) {
        const int tiles_t = (d.T + 255) / 256;
        a.rows_t = ((d.T + tiles_t - 1) / tiles_t + 15) / 16 * 16;
        const int per_tile = a.gated ? 64 : 128;
        const int tiles_n = (d.N + per_tile - 1) / per_tile;
        const int stage = kLinA + a.rows_t * 128;
        a.stages = a.rows_t <= 32 ? 4 : a.rows_t <= 96 ? 4 : 4;
        if (!encode16(&m.x, x, d.K, d.T, d.ldx, a.rows_t) ||
            !encode16(&m.w, w, d.K, d.N, d.ldw, per_tile) ||
            (a.gated && !encode16(&m.v, w_mul, d.K, d.N, d.ldw, per_tile)))
            return cudaErrorInvalidValue;
        int splits = 1;
        while (splits < 8 && 2 * splits <= a.nk && (int64_t)tiles_n * tiles_t * splits * 2 <= 2 * sms) splits *= 2;
        return launch_clusters(linear_few_kernel, dim3(tiles_n * splits, tiles_t), splits, kFewThreads,
                               a.stages * stage + 1024, m, a, st);
    }
    // TMA addresses rows that start at multiples of 16 bytes
    a.tma_rows = rows_aligned(out, d.ldo, 16) && (!residual || rows_aligned(residual, d.ldr, 16));
    if (!encode16(&m.x, x, d.K, d.T, d.ldx, 128) || !encode16(&m.w, w, d.K, d.N, d.ldw, 64) ||
        (a.gated && !encode16(&m.v, w_mul, d.K, d.N, d.ldw, 64)) ||
        (a.tma_rows && !encode16(&m.out, out, d.N, d.T, d.ldo, 128)) ||
        (a.tma_rows && residual && !encode16(&m.res, residual, d.N, d.T, d.ldr, 128)))
        return cudaErrorInvalidValue;
    a.wave = sms / 2;
    const int64_t total = ManySched(d.T, d.N, a.gated, a.wave).total;
    const int pairs = (int)(total < a.wave ? total : a.wave);
    return launch_clusters(linear_many_kernel, dim3(2 * pairs), 2, kManyThreads, kManySmem, m, a, st);
}

}  // namespace moe
