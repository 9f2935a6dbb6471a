// adapters.cu -- the low-rank products of moe_linear_adapters: v[t] = scale[j] x[t] a[j]^T, j = ids[t].
//
// Rows are taken in groups of 256.  In a group the rows of one adapter form batches of up to 32 in their order,
// and an item is a batch and 32 of the stacked ranks (both matrices' in the gated form): D = A x^T by mma.sync,
// ranks on the M side, rows of x on the N side (8 where the batch has no more, or 32).  Each byte of a that a batch needs
// is read once for all of its rows, in 16-byte loads straight into the fragments: the sum may take K in any
// order, so a lane's four 16-bit pairs of one 16-byte load serve as the operands of two MMAs, the same way on both sides.
// K is split over the warps of a CTA and the CTAs of a cluster; the parts meet in shared memory and are added in
// order.  A batch of one token costs its adapter's bytes, a prompt's its rows of x, read here before the layer
// reads them again from L2.  tcgen05 would take 128 lanes for 16 to 64 ranks.
//
// Which adapters occur is known on the device alone: every CTA of a group finds the batches by itself (a comparison
// with the ids before it per row), so that no launch has to sort them.
//
// How v is held, and what becomes of a v that the layer's type does not hold: kernels.h.
//
// Alone and cold, 1 gated row of 7168, rank 16: 7 to 9 us, latency; 512 rows of 2048 with 32 adapters: 11 us; 4096 gated rows of 7168:
// 22 us; 16384 rows of 2048, rank 64: 55 us, the loads of x for every 32 ranks and of a for every 32 rows from L2.  A whole call
// with the layer: 17.0 us for that one row, 37.8 for 64 gated rows of 4096 with an adapter each, 179 for those 4096, 351 for the
// 16384.  The 128 registers that two CTAs to an SM leave do not hold all: 56 bytes of spills beside the sums.
#include "cluster.cuh"
#include "kernels.h"
#include "launch_plan.h"
#include "tc_ptx.cuh"
#include "rows.cuh"

namespace moe {

namespace {

constexpr int kGroup = kLowGroup, kBatch = kLowBatch, kRanks = kLowRanks;

struct LowRankArgs {
    int T, K, R, L, f16, matrices, slots, landing_rows;  // landing_rows: of a batch at most
    int64_t ldx, lda, sa, plane, far_plane, marks_plane;  // elements of a plane of v, of far and of marks
    const uint16_t *x, *a[2];
    const float* scale;
    const int32_t* ids;
    float* whole;  // v as it is; or nullptr, and v in two numbers
    uint16_t* v;
    float* far;
    uint8_t* marks;
    int32_t* status;
};

template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (F16) mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
    else mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
}

// This warp's part of an item's sums, over the steps of 32 elements of K from `step` on, `stride` apart: NB blocks of 8
// rows.  With g = lane / 4, rank: where the item's ranks g, g + 8, g + 16 and g + 24 of a begin, row: where the batch's rows g, g + 8,
// ... of x do (nullptr: none).
template <bool F16, int NB, int UNROLL>
__device__ __forceinline__ void low_rank_sums(float (&d)[2][4][4], const uint16_t* const (&rank)[4],
                                              const uint16_t* const (&row)[4], int step, int stride, int end, int K) {
    const int c8 = 8 * (threadIdx.x & 3);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (; step < end; step += UNROLL * stride) {
        uint4 w[UNROLL][4], x[UNROLL][NB];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int k = 32 * (step + u * stride) + c8;
            const bool in = step + u * stride < end && k < K;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[u][i] = in && rank[i] ? __ldcg(reinterpret_cast<const uint4*>(rank[i] + k)) : zero;
#pragma unroll
            for (int i = 0; i < NB; ++i) x[u][i] = in && row[i] ? __ldcg(reinterpret_cast<const uint4*>(row[i] + k)) : zero;
        }
        __syncwarp();  // the MMAs want the whole warp, and the loads above may part it
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const uint4 p = w[u][2 * m], q = w[u][2 * m + 1];
                    mma16<F16>(d[m][i], p.x, q.x, p.y, q.y, x[u][i].x, x[u][i].y);
                    mma16<F16>(d[m][i], p.z, q.z, p.w, q.w, x[u][i].z, x[u][i].w);
                }
    }
}

// grid (slots * CTAs of a cluster, groups): slot s takes the group's items s, s + slots, ... in parts of K by its CTAs; where
// a group has more items than slots, each CTA takes whole items of its own.
template <bool F16>
__global__ void __launch_bounds__(kGroup, 2) low_rank_kernel(LowRankArgs g) {
    __shared__ __align__(16) int id_s[kGroup];
    __shared__ int batch_row[kBatch], leaders[kGroup / 32], item_id, item_first;
    __shared__ __align__(16) float part[4][kBatch][kRanks + 4];     // sums of a warp: [row][rank]
    extern __shared__ __align__(16) float landing[];                // [CTA][row][rank]
    pdl_wait();
    pdl_trigger();  // the layer's launch may start: whatever came before this one is done
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cluster = (int)cluster_size();
    if (cluster > 1) cluster_arrive();  // this CTA runs: its shared memory may be written from the others
    const int64_t t0 = (int64_t)blockIdx.y * kGroup;
    int id = t0 + tid < g.T ? __ldcg(g.ids + t0 + tid) : -1;
    if (id < -1 || id >= g.L) {
        if (blockIdx.x == 0) status_or(g.status, MOE_DEV_BAD_ADAPTER_ID);
        id = -1;
    }
    id_s[tid] = id;
    __syncthreads();
    int before = 0;  // rows of this adapter before this one
    if (id >= 0) {
        for (int i = 0; i < (tid & ~3); i += 4) {
            const int4 p = *reinterpret_cast<const int4*>(id_s + i);
            before += (p.x == id) + (p.y == id) + (p.z == id) + (p.w == id);
        }
        for (int i = tid & ~3; i < tid; ++i) before += id_s[i] == id;
    }
    const bool leads = id >= 0 && before % kBatch == 0;
    const unsigned lead_mask = __ballot_sync(0xffffffffu, leads);
    if (lane == 0) leaders[warp] = __popc(lead_mask);
    __syncthreads();
    int batches = 0, batch = __popc(lead_mask & ((1u << lane) - 1u));  // of the group; the one this row leads
#pragma unroll
    for (int w = 0; w < kGroup / 32; ++w) {
        if (w < warp) batch += leaders[w];
        batches += leaders[w];
    }
    const int per_matrix = (g.R + 15) / 16, passes = (per_matrix * g.matrices + 1) / 2;  // blocks of 16 ranks, items of a batch
    const int steps = (g.K + 31) / 32;
    const int ctas = batches * passes > g.slots ? 1 : cluster, cta = ctas > 1 ? (int)cluster_rank() : 0;  // of an item
    const int begin = (int)((int64_t)steps * cta / ctas), end = (int)((int64_t)steps * (cta + 1) / ctas);
    if (cluster > 1) cluster_wait();
    for (int item = (int)blockIdx.x / ctas; item < batches * passes; item += (int)gridDim.x / ctas) {
        const int pass = item % passes;
        if (leads && batch == item / passes) {
            item_id = id;
            item_first = before;
        }
        __syncthreads();
        const int j = item_id, first = item_first;
        const bool here = id == j && before >= first && before < first + kBatch;
        if (here) batch_row[before - first] = tid;
        const int rows = __syncthreads_count(here);
        const uint16_t *rank[4], *row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int block = 2 * pass + (i >> 1), m = block >= per_matrix, r = 16 * (block - m * per_matrix) + 8 * (i & 1) + (lane >> 2);
            rank[i] = block < per_matrix * g.matrices && r < g.R ? g.a[m] + j * g.sa + r * g.lda : nullptr;
            row[i] = 8 * i + (lane >> 2) < rows ? g.x + (t0 + batch_row[8 * i + (lane >> 2)]) * g.ldx : nullptr;
        }
        float d[2][4][4] = {};
        if (rows <= 8) low_rank_sums<F16, 1, 4>(d, rank, row, begin + warp, kGroup / 32, end, g.K);
        else low_rank_sums<F16, 4, 2>(d, rank, row, begin + warp, kGroup / 32, end, g.K);
        const int blocks = rows <= 8 ? 1 : 4;
        // warps 4 to 7 hand theirs to warps 0 to 3, these add them to their own, and those four are added
        const auto place = [&](int m, int b, int e) -> float& {
            return part[warp & 3][8 * b + 2 * (lane & 3) + (e & 1)][16 * m + (lane >> 2) + 8 * (e >> 1)];
        };
        const auto each = [&](auto&& f) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (b < blocks) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) f(d[m][b][e], place(m, b, e));
                    }
        };
        if (warp >= 4) each([](float v, float& at) { at = v; });
        __syncthreads();
        if (warp < 4) each([](float v, float& at) { at = v + at; });
        __syncthreads();
        // a thread: one row of the batch (of 32), four ranks
        const int at_row = tid >> 3, at_rank = 4 * (tid & 7);
        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        if (at_row < rows)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 p = *reinterpret_cast<const float4*>(&part[w][at_row][at_rank]);
                z.x += p.x; z.y += p.y; z.z += p.z; z.w += p.w;
            }
        if (ctas > 1) {
            const uint32_t there = tc::smem_u32(landing + (cta * g.landing_rows + at_row) * kRanks + at_rank);
            if (at_row < rows)
                st_cluster_v4(map_rank(there, 0), __float_as_uint(z.x), __float_as_uint(z.y), __float_as_uint(z.z), __float_as_uint(z.w));
            cluster_sync();
            if (cta == 0 && at_row < rows) {
                z = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c = 0; c < ctas; ++c) {
                    const float4 p = *reinterpret_cast<const float4*>(landing + (c * g.landing_rows + at_row) * kRanks + at_rank);
                    z.x += p.x; z.y += p.y; z.z += p.z; z.w += p.w;
                }
            }
        }
        const int block = 2 * pass + (at_rank >> 4), m = block >= per_matrix, r = 16 * (block - m * per_matrix) + (at_rank & 15);
        // R is a multiple of 8: all four ranks or none
        const bool mine = cta == 0 && at_row < rows && block < per_matrix * g.matrices && r < g.R;
        const float s = g.scale ? __ldcg(g.scale + j) : 1.f;
        const float v[4] = {z.x * s, z.y * s, z.z * s, z.w * s};
        const int64_t t = mine ? t0 + batch_row[at_row] : 0;
        if (g.whole) {
            if (mine) *reinterpret_cast<float4*>(g.whole + m * g.plane + t * g.R + r) = make_float4(v[0], v[1], v[2], v[3]);
            if (ctas > 1) cluster_sync();  // the landing area is free
            __syncthreads();               // and the batch's rows
            continue;
        }
        float far[4] = {};
        uint16_t hi[4], lo[4];
        bool beyond = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F16) {
                const __half h = __float2half_rn(v[i]);
                hi[i] = __half_as_ushort(h);
                lo[i] = __half_as_ushort(__float2half_rn(v[i] - __half2float(h)));
            } else {
                const __nv_bfloat16 h = __float2bfloat16_rn(v[i]);
                hi[i] = __bfloat16_as_ushort(h);
                lo[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v[i] - __bfloat162float(h)));
            }
            constexpr uint16_t kInf = F16 ? 0x7C00u : 0x7F80u;
            if ((hi[i] & kInf) == kInf) {  // the type does not hold it
                beyond = mine;
                far[i] = v[i];
                hi[i] = lo[i] = 0;
            }
        }
        // the four lanes of a block of 16 ranks stand side by side
        const bool marked = (__ballot_sync(0xffffffffu, beyond) >> (lane & 28)) & 15u;
        if (mine) {
            uint16_t* to = g.v + 2 * m * g.plane + t * g.R + r;
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16);
            *reinterpret_cast<uint2*>(to + g.plane) = make_uint2(lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16);
            if (marked) *reinterpret_cast<float4*>(g.far + m * g.far_plane + t * g.R + r) = make_float4(far[0], far[1], far[2], far[3]);
            if (r % kFarRanks == 0) g.marks[m * g.marks_plane + t * kFarMarks + r / kFarRanks] = marked;
        }
        if (ctas > 1) cluster_sync();  // the landing area is free
        __syncthreads();               // and the batch's rows
    }
}

template <bool F16>
cudaError_t launch_low_rank(const LowRankArgs& g, int groups, int splits, int smem, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(g.slots * splits), (unsigned)groups);
    cfg.blockDim = dim3(kGroup);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, low_rank_kernel<F16>, g);
}

}  // namespace

cudaError_t launch_linear_adapters(const moe_linear_desc& d, const moe_adapter_desc& ad, const void* x, const void* w,
                                   const void* w_mul, const float* bias, const float* bias_mul, const void* residual,
                                   void* out, void* workspace, int32_t* status, cudaStream_t st) {
    LinPlan layer;
    const cudaError_t planned = plan_layer(d, w_mul != nullptr, layer);
    if (planned != cudaSuccess) return planned;
    const AdapterProducts p = AdapterProducts::plan(d.T, ad.R, ad.a && ad.a_mul ? 2 : 1);
    LowRankArgs g{};
    g.T = d.T; g.K = d.K; g.R = ad.R; g.L = ad.L; g.f16 = d.dtype == MOE_DT_F16; g.matrices = p.matrices;
    g.ldx = d.ldx; g.lda = ad.lda; g.sa = ad.sa;
    g.plane = (int64_t)(p.plane / sizeof(uint16_t)); g.far_plane = (int64_t)(p.far_plane / sizeof(float)); g.marks_plane = (int64_t)p.marks_plane;
    g.x = static_cast<const uint16_t*>(x);
    g.a[0] = static_cast<const uint16_t*>(ad.a ? ad.a : ad.a_mul);
    g.a[1] = static_cast<const uint16_t*>(ad.a_mul);
    g.scale = ad.scale; g.ids = ad.ids;
    g.whole = layer.few ? static_cast<float*>(workspace) : nullptr;
    g.v = static_cast<uint16_t*>(workspace);
    g.far = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.far);
    g.marks = static_cast<uint8_t*>(workspace) + p.marks;
    g.status = status;
    const LowPlan plan = plan_low_rank(d.T, d.K, ad.L, ad.R, p.matrices);
    g.slots = plan.slots;
    g.landing_rows = plan.landing_rows;
    // groups are the grid's second dimension: at most 65535 a launch
    for (int first = 0; first < plan.groups; first += 65535) {
        const int n = plan.groups - first < 65535 ? plan.groups - first : 65535;
        LowRankArgs h = g;
        const int64_t t = (int64_t)first * kGroup;
        h.x += t * g.ldx;
        h.ids += t;
        if (h.whole) h.whole += t * g.R;
        h.v += t * g.R;
        h.far += t * g.R;
        h.marks += t * kFarMarks;
        h.T = (int)(g.T - t);
        const cudaError_t err = g.f16 ? launch_low_rank<true>(h, n, plan.splits, plan.smem, st) : launch_low_rank<false>(h, n, plan.splits, plan.smem, st);
        if (err != cudaSuccess) return err;
    }
    return launch_adapted_linear(layer, d, ad, x, w, w_mul, bias, bias_mul, residual, out, workspace, status, st);
}

}  // namespace moe
