// adapters.cu -- the low-rank products of moe_linear_adapters: v[t] = scale[j] x[t] a[j]^T, j = ids[t].
//
// Rows are taken in groups of 128.  A group's adapters, in the order in which they first occur, have their ranks (both
// matrices' in the gated form) stacked in units of 16 to 128, and a tile is up to 128 of these ranks, the rows of a
// tcgen05.mma.kind::f16 whose columns are the group's rows of x: D = A x^T.  What a row needs of it are the units of its own
// adapter; the rest is left out (a product costs its operands' way to the SM, and each of them comes once: an adapter's bytes
// for a token, the rows of x for a prompt).  Both come by TMA, a unit as one box, through warps of their own (one thread
// took 350 ns for a stage of two boxes); x starts while the adapters are found.  K is split over the CTAs of a cluster, which exchange the products that count through distributed
// shared memory and add them in rank order.
//
// Which adapters occur is known on the device alone.  Every CTA finds its group's by itself: a row leads if no row
// before it has its adapter, and the leaders before it number it.
#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"
#include "launch_plan.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

using namespace tc;

struct LowMaps {
    CUtensorMap x, a[2];
};
struct LowArgs {
    int T, R, L, matrices, steps, f16;  // steps of K in all
    int rows, own_log2, unit_log2, per_adapter_log2, tile, width, slots, stages, stage, loaders;
    int64_t plane;  // elements of 16 bits
    const float* scale;
    const int32_t* ids;
    uint16_t* v;
    int32_t* status;
};
constexpr int kLowThreads = 256;
static_assert(kLowThreads / 32 - 2 == kLowLoaders);

// kind::f16: fp32 D of 128 rows, A and B both bf16 (format 1) or both f16 (format 0), K-major.
__device__ __forceinline__ uint32_t low_idesc(uint32_t N, bool f16) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | ((N >> 3) << 17) | (8u << 24);
}

// grid (CTAs of a cluster, groups, slots): slot s takes the group's tiles s, s + slots, ...
__global__ void __launch_bounds__(kLowThreads, 1)
low_rank_kernel(const __grid_constant__ LowMaps maps, const __grid_constant__ LowArgs g) {
    extern __shared__ uint8_t low_smem[];
    __shared__ uint64_t full[kLowStages], empty[kLowStages], acc_full;
    __shared__ __align__(16) int id_s[kLowRows];  // of the rows, then of the adapters in their order
    __shared__ __align__(16) int8_t place[kLowRows];  // of a row's adapter in that order
    __shared__ int leaders[kLowRows / 32];
    __shared__ uint32_t tmem_slot;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(low_smem) + 1023) & ~uintptr_t(1023));
    float* landing = reinterpret_cast<float*>(smem + g.stages * g.stage);  // [CTA][own row][rank of its adapter in the tile]
    float* scale_s = landing + ((int)cluster_size() << g.own_log2) * g.width;           // of the adapters in their order
    const int warp = warp_index(), lane = threadIdx.x & 31, tid = threadIdx.x;
    const int ctas = (int)cluster_size(), cta = (int)cluster_rank();
    const int64_t t0 = (int64_t)blockIdx.y * g.rows;
    const int ncols = (int)min((int64_t)g.rows, g.T - t0);
    const int k_begin = (int)((int64_t)g.steps * cta / ctas), steps = (int)((int64_t)g.steps * (cta + 1) / ctas) - k_begin;
    const int unit = 1 << g.unit_log2, own = 1 << g.own_log2;
    const int x_at = g.tile * unit * 128;  // of a stage
    uint32_t tm_cols = kTmemLeast;
    while ((int)tm_cols < g.rows) tm_cols *= 2;
    if (tid == 0) {
        for (int s = 0; s < g.stages; ++s) {
            mbar_init(&full[s], 1 + g.tile);  // x, and every unit
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        fence_mbar_init();
        prefetch_tmap(&maps.x);
        prefetch_tmap(&maps.a[0]);
        if (g.matrices == 2) prefetch_tmap(&maps.a[1]);
    }
    if (warp == 1) tmem_alloc(&tmem_slot, tm_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    cluster_arrive();  // this CTA runs: its shared memory may be written from the others
    pdl_wait();
    // The layer's launch may start: whatever came before this one is done.  (Once the first loads are here, so that they are
    // not behind the layer's: 8 rows 16.6 us for 12.4.)
    pdl_trigger();
    auto give_up = [&]() { status_or(g.status, MOE_DEV_TIMEOUT); };
    const auto load_x = [&](int s, int i) {
        mbar_arrive_expect_tx(&full[s], g.rows * 128);
        tma_load_2d(smem + s * g.stage + x_at, &maps.x, (k_begin + i) * kLowK, (int)t0, &full[s]);
    };
    // roles of elected lanes as in linear.cu: the rest of their warps waits at the end of the role
    const int ahead = min(steps, g.stages);  // stages whose x comes before the adapters are known
    if (warp >= kLowRows / 32) {  // the others find the adapters meanwhile
        if (elect_one())
            for (int i = warp - kLowRows / 32; i < ahead; i += kLowThreads / 32 - kLowRows / 32) load_x(i, i);
        __syncwarp();
    }
    // the group's adapters
    int id = -1;
    float scale = 1.f;
    if (tid < kLowRows) {
        if (tid < ncols) id = __ldg(g.ids + t0 + tid);
        if (id < -1 || id >= g.L) {
            if (blockIdx.x == 0 && blockIdx.z == 0) status_or(g.status, MOE_DEV_BAD_ADAPTER_ID);
            id = -1;
        }
        id_s[tid] = id;
        if (g.scale && id >= 0) scale = __ldg(g.scale + id);
    }
    __syncthreads();
    // the first row that has this row's adapter: of its warp's, or of those before
    int first = (tid & ~31) + __ffs(__match_any_sync(0xffffffffu, id)) - 1;
    if (tid < kLowRows) {
        bool found = id < 0;
        for (int i = 0; i < (tid & ~31) && !__all_sync(0xffffffffu, found); i += 4) {
            const int4 p = *reinterpret_cast<const int4*>(id_s + i);
            const int at = p.x == id ? 0 : p.y == id ? 1 : p.z == id ? 2 : 3;
            if (!found && (at < 3 || p.w == id)) {
                first = i + at;
                found = true;
            }
        }
    }
    const bool leads = id >= 0 && first == tid;
    const unsigned lead_mask = __ballot_sync(0xffffffffu, leads);
    if (lane == 0 && warp < kLowRows / 32) leaders[warp] = __popc(lead_mask);
    __syncthreads();
    int adapters = 0, number = __popc(lead_mask & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kLowRows / 32; ++w) {
        if (w < warp) number += leaders[w];
        adapters += leaders[w];
    }
    if (leads) {
        id_s[number] = id;
        place[tid] = (int8_t)number;
    }
    __syncthreads();
    if (tid < kLowRows && !leads) place[tid] = id >= 0 ? place[first] : (int8_t)-1;
    const int per_adapter = 1 << g.per_adapter_log2, units = adapters << g.per_adapter_log2, per_matrix = per_adapter / g.matrices;
    const int my_c0 = cta * own, my_cols = min(own, ncols - my_c0);  // this CTA's rows of x
    int done = 0;  // tiles
    for (int tile = blockIdx.z; tile * g.tile < units; tile += g.slots, ++done) {
        const int u0 = tile * g.tile, here = min(g.tile, units - u0);
        RingPos ring;  // `done` tiles of `steps` stages on
        ring.slot = (done * steps) % g.stages;
        ring.parity = (uint32_t)((done * steps) / g.stages) & 1u;
        if (warp == 0) {
            if (elect_one()) {
                int i = 0;
                RingPos at = ring;
                for (; i < steps; ++i, at.next(g.stages)) {
                    if (done == 0 && i < ahead) continue;
                    if (!mbar_wait_suspended(&empty[at.slot], at.parity ^ 1)) {
                        give_up();
                        break;
                    }
                    load_x(at.slot, i);
                }
                // whoever gives up, no copy is in flight when the CTA ends
                for (int left = i < g.stages ? i : g.stages; left > 0; --left) {
                    at.back(g.stages);
                    mbar_wait_suspended(&full[at.slot], at.parity);
                }
            }
            __syncwarp();
        } else if (warp >= 2) {
            // Units of stages in turn, so that all loaders have some however few units there are; a unit that a short tile
            // lacks arrives without bytes.  A loader goes on by a lap of the ring at most: a barrier's parity tells the
            // lap before from this one, not from the one before that.
            if (warp - 2 < g.loaders && elect_one()) {
                RingPos at = ring;
                int i = 0;  // stage
                for (int k = warp - 2;; k += g.loaders) {
                    for (; k >= g.tile; k -= g.tile) {
                        ++i;
                        at.next(g.stages);
                    }
                    if (i >= steps) break;
                    if (!mbar_wait_suspended(&empty[at.slot], at.parity ^ 1)) {
                        give_up();
                        break;
                    }
                    uint64_t* const bar = &full[at.slot];
                    mbar_arrive_expect_tx(bar, k < here ? unit * 128 : 0);
                    if (k >= here) continue;
                    const int of = (u0 + k) >> g.per_adapter_log2, u = (u0 + k) & (per_adapter - 1), second = u >= per_matrix;
                    tma_load_3d(smem + at.slot * g.stage + k * unit * 128, &maps.a[second], (k_begin + i) * kLowK,
                                (u - (second ? per_matrix : 0)) << g.unit_log2, id_s[of], bar);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            if (elect_one()) {
                const uint32_t idesc = low_idesc((uint32_t)g.rows, g.f16);
                RingPos at = ring;
                for (int i = 0; i < steps; ++i, at.next(g.stages)) {
                    const int s = at.slot;
                    if (!mbar_wait_suspended(&full[s], at.parity)) {
                        give_up();
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc(smem_u32(smem + s * g.stage), 16, 1024, kLayoutSw128);
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // K 16 per MMA: 32 bytes (two units) along the swizzled row
                        tc_mma_bf16(tmem, ad + 2 * j, ad + (x_at >> 4) + 2 * j, idesc, (i | j) != 0);
                    tc_commit(&empty[s]);
                }
                tc_commit(&acc_full);  // arrives when every MMA has completed
                if (!mbar_wait_suspended(&acc_full, (uint32_t)done & 1u)) give_up();
                tc_fence_before();
            }
            __syncwarp();
        }
        if (done == 0) {
            if (leads) scale_s[number] = scale;  // not before: nobody waits for its load until now
            cluster_wait();
        }
        __syncthreads();  // all wait here for that
        {  // A lane is a rank; the two warps of a lane quarter take alternate 32 columns, of those, by fours, the ones with an adapter
           // of this tile: two or three of 64 tokens with one each, all of a prompt.
            tc_fence_after();
            const int q = warp & 3, u = u0 + ((32 * q + lane) >> g.unit_log2), of = u >> g.per_adapter_log2;  // adapter of the lane
            const int rank = 32 * q + lane - ((max(of << g.per_adapter_log2, u0) - u0) << g.unit_log2);       // of those of that adapter here
            const int mine = u < u0 + here ? of : kLowRows;
            const int low = u0 >> g.per_adapter_log2, high = (u0 + here - 1) >> g.per_adapter_log2;  // adapters of the tile
            const uint32_t to = smem_u32(landing + (cta << g.own_log2) * g.width + rank);
            for (int c0 = 32 * (warp >> 2); 32 * q < here * unit && c0 < ncols; c0 += 64) {
                const int at = place[c0 + lane];
                const unsigned has = __ballot_sync(0xffffffffu, at >= low && at <= high);
#pragma unroll 1
                for (int i = 0; i < 32; i += 4) {  // four columns at a time, where one of them has
                    if (!(has >> i & 15u)) continue;
                    const int c = c0 + i;
                    uint32_t v[4];
                    tmem_ld_4(tmem + ((uint32_t)(32 * q) << 16) + c, v);
                    const uint32_t there = map_rank(to + (c & (own - 1)) * g.width * 4, c >> g.own_log2);  // own is a multiple of four
                    const uint32_t places = *reinterpret_cast<const uint32_t*>(place + c);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if ((int)(places >> (8 * k) & 0xFFu) == mine) st_cluster(there + k * g.width * 4, v[k]);
                    __syncwarp();
                }
            }
            tc_fence_before();
        }
        cluster_sync();  // every part has landed
        const int fours_log2 = 29 - __clz(g.width);  // width is a power of two
        for (int i = tid; i < my_cols << fours_log2; i += kLowThreads) {  // a row's four ranks
            const int c = i >> fours_log2, n = 4 * (i & ((1 << fours_log2) - 1)), of = place[my_c0 + c];
            const int from = max(of << g.per_adapter_log2, u0), end = min((of + 1) << g.per_adapter_log2, u0 + g.tile);  // its units here
            if (of < 0 || n >= (end - from) << g.unit_log2) continue;
            const int u = from - (of << g.per_adapter_log2) + (n >> g.unit_log2), m = u >= per_matrix;  // of the adapter
            const int r = ((u - (m ? per_matrix : 0)) << g.unit_log2) + (n & (unit - 1));
            if (r >= g.R) continue;  // R is a multiple of 8: all four or none
            const float* src = landing + c * g.width + n;
            float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < kLowSplits; ++s)
                if (s < ctas) {
                    const float4 p = *reinterpret_cast<const float4*>(src + (s << g.own_log2) * g.width);
                    z.x += p.x; z.y += p.y; z.z += p.z; z.w += p.w;
                }
            const float times = scale_s[of];
            const float v[4] = {z.x * times, z.y * times, z.z * times, z.w * times};
            uint16_t* const to_v = g.v + 2 * m * g.plane;
            const int64_t at = (t0 + my_c0 + c) * g.R + r;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // an infinite hi has no rest
                if (g.f16) {
                    const __half h = __float2half_rn(v[k]);
                    hi[k] = __half_as_ushort(h);
                    lo[k] = (hi[k] & 0x7C00u) == 0x7C00u ? 0 : __half_as_ushort(__float2half_rn(v[k] - __half2float(h)));
                } else {
                    const __nv_bfloat16 h = __float2bfloat16_rn(v[k]);
                    hi[k] = __bfloat16_as_ushort(h);
                    lo[k] = (hi[k] & 0x7F80u) == 0x7F80u ? 0 : __bfloat16_as_ushort(__float2bfloat16_rn(v[k] - __bfloat162float(h)));
                }
            }
            *reinterpret_cast<uint2*>(to_v + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(to_v + g.plane + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        }
        if ((tile + g.slots) * g.tile < units) cluster_sync();  // the landing areas and tensor memory are free
    }
    if (done == 0) cluster_wait();
    if (done == 0 && warp == 0) {  // nothing used the x that came ahead
        if (elect_one())
            for (int i = 0; i < ahead; ++i) {
                for (int k = 0; k < g.tile; ++k) mbar_arrive(&full[i]);
                mbar_wait_suspended(&full[i], 0);
            }
        __syncwarp();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, tm_cols);
    }
}

}  // namespace

cudaError_t launch_linear_adapters(const moe_linear_desc& d, const moe_adapter_desc& ad, const void* x, const void* w,
                                   const void* w_mul, const float* bias, const float* bias_mul, const void* residual,
                                   void* out, void* workspace, int32_t* status, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    static std::atomic<uint64_t> allowed{0};
    if (err == cudaSuccess) err = allow_large_launch(low_rank_kernel, kCtaSmemMax, allowed);
    if (err != cudaSuccess) return err;
    const AdapterProducts products = AdapterProducts::plan(d.T, ad.R, ad.a && ad.a_mul ? 2 : 1);
    const LowPlan p = plan_low_rank(d.T, d.K, ad.L, ad.R, products.matrices, sms);
    const void* of[2] = {ad.a ? ad.a : ad.a_mul, products.matrices == 2 ? ad.a_mul : nullptr};
    LowMaps m{};
    if (!encode_rows16(&m.x, x, d.K, d.T, d.ldx, p.rows, kLowK)) return cudaErrorInvalidValue;
    for (int i = 0; i < products.matrices; ++i)
        if (!encode_stack16(&m.a[i], of[i], d.K, ad.R, ad.L, ad.lda, ad.L > 1 ? ad.sa : ad.R * ad.lda, 1 << p.unit_log2, kLowK)) return cudaErrorInvalidValue;
    LowArgs g{};
    g.T = d.T; g.R = ad.R; g.L = ad.L; g.matrices = products.matrices; g.steps = (d.K + kLowK - 1) / kLowK; g.f16 = d.dtype == MOE_DT_F16;
    g.rows = p.rows; g.own_log2 = p.own_log2; g.unit_log2 = p.unit_log2; g.tile = p.tile; g.width = p.width; g.per_adapter_log2 = p.per_adapter_log2; g.slots = p.slots; g.stages = p.stages; g.stage = p.stage; g.loaders = p.loaders;
    g.plane = (int64_t)(products.plane / 2);
    g.scale = ad.scale; g.ids = ad.ids; g.v = static_cast<uint16_t*>(workspace); g.status = status;
    // groups are the grid's second dimension: at most 65535 a launch
    for (int first = 0; first < p.groups; first += 65535) {
        const int n = p.groups - first < 65535 ? p.groups - first : 65535;
        const int64_t t = (int64_t)first * p.rows;
        LowArgs h = g;
        if (first) {
            if (!encode_rows16(&m.x, static_cast<const uint16_t*>(x) + t * d.ldx, d.K, d.T - t, d.ldx, p.rows, kLowK)) return cudaErrorInvalidValue;
            h.T = (int)(d.T - t);
            h.ids += t;
            h.v += t * g.R;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)p.splits, (unsigned)n, (unsigned)p.slots);
        cfg.blockDim = dim3(kLowThreads);
        cfg.dynamicSmemBytes = p.smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)p.splits;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        err = cudaLaunchKernelEx(&cfg, low_rank_kernel, m, h);
        if (err != cudaSuccess) return err;
    }
    return launch_adapted_linear(d, ad, x, w, w_mul, bias, bias_mul, residual, out, workspace, status, st);
}

}  // namespace moe
