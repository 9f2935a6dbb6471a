// block_norm.cu -- the norms behind a block and before the next one, with the gate and the residual between:
// p = y / sqrt(mean(y^2) + eps) * (post_weight + offset), s = residual_scale r + g p,
// n = s / sqrt(mean(s^2) + eps) * (weight + offset).
//
// A CTA per row, or a warp per row for short ones.  The row stays in registers through both sums of squares, so
// every input is read once and every output written once, where two kernels would read s again.  The weights,
// the same for every row, are read between the sums, when they come from L1 or L2 and the row's inputs no longer
// take registers.  p, s, their squares and the scalings are fp32; s and n are each rounded once, n from the
// unrounded s.
#include "kernels.h"
#include "rows.cuh"

namespace moe {

namespace {

struct BlockNormArgs {
    const void *y, *r, *post, *gate, *w;
    const float* row_gate;
    void *sum, *out;
    int64_t ldy, ldr, lds, ldo;
    int T, H, sigmoid;
    float eps, scale, offset;
};

// The sum of v over the row's threads: a warp's, or the CTA's through `part`.
template <int WARPS>
__device__ __forceinline__ float row_sum(float v, float* part, int lane, int warp) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (!WARPS) {
        if (lane == 0) part[warp] = v;
        __syncthreads();
        v = lane < (blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// WARPS: rows per CTA, a warp each; 0: one row per CTA, by all its warps.  S: type of r and s.
template <typename E, typename S, int MODE, int VPT, int WARPS>
__global__ void __launch_bounds__(WARPS ? 32 * WARPS : 1024, !WARPS && VPT == 1 ? 2 : 1)
sandwich_norm_kernel(BlockNormArgs a) {
    constexpr int VEC = MODE == ROWS_SINGLE ? 1 : 8;
    using P = Pack<E, VEC>;
    using Q = Pack<S, VEC>;
    __shared__ float part[2][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = WARPS ? (int64_t)blockIdx.x * WARPS + warp : blockIdx.x;
    if (WARPS && t >= a.T) return;
    const int tid = WARPS ? lane : threadIdx.x, step = WARPS ? 32 : blockDim.x;
    const E* y = static_cast<const E*>(a.y) + t * a.ldy;
    const S* r = a.r ? static_cast<const S*>(a.r) + t * a.ldr : nullptr;
    S* sum = static_cast<S*>(a.sum) + t * a.lds;
    E* out = a.out ? static_cast<E*>(a.out) + t * a.ldo : nullptr;
    // elements between the boundary before the row and its start (the same for all tensors)
    const int off = MODE == ROWS_SHIFTED ? (int)((reinterpret_cast<uintptr_t>(y) >> 1) & 7) : 0;
    const int nvec = (a.H + off + VEC - 1) / VEC;
    const auto weights = [&](const void* w, int c0) {
        if constexpr (MODE == ROWS_SHIFTED) return load_weight<E>(static_cast<const E*>(w), c0, a.H);
        else return *reinterpret_cast<const P*>(static_cast<const E*>(w) + c0);
    };
    P yv[VPT];
    Q rv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {  // every load of the row issued before any is used
        const int c = tid + i * step, c0 = c * VEC - off;
        if (c < nvec) {
            yv[i] = load_vec<E, MODE, VEC>(y, c0, a.H);
            if (r) rv[i] = load_vec<S, MODE, VEC>(r, c0, a.H);
        }
    }
    float g = a.row_gate ? __ldcg(a.row_gate + t) : 1.f;
    if (a.sigmoid) g = 1.f / (1.f + __expf(-g));
    if (a.post) {
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (tid + i * step < nvec) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float v = to_f32(yv[i].v[j]);  // elements outside the row are 0
                    sq += v * v;
                }
            }
        g *= rsqrtf(row_sum<WARPS>(sq, part[0], lane, warp) / (float)a.H + a.eps);
    }
    float s[VPT][VEC], sq = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * step, c0 = c * VEC - off;
        if (c < nvec) {
            Q o;
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[i][j] = to_f32(yv[i].v[j]) * g;
            if (a.post) {
                const P w = weights(a.post, c0);
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[i][j] *= to_f32(w.v[j]) + a.offset;
            }
            if (a.gate) {
                const P w = weights(a.gate, c0);
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[i][j] *= to_f32(w.v[j]);
            }
            if (r) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[i][j] += a.scale * to_f32(rv[i].v[j]);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                sq += s[i][j] * s[i][j];
                from_f32(s[i][j], o.v[j]);
            }
            store_vec<S, MODE, VEC>(sum, c0, a.H, o);
        }
    }
    if (!out) return;
    const float scale = rsqrtf(row_sum<WARPS>(sq, part[1], lane, warp) / (float)a.H + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * step, c0 = c * VEC - off;
        if (c < nvec) {
            const P w = weights(a.w, c0);
            P o;
#pragma unroll
            for (int j = 0; j < VEC; ++j) from_f32(s[i][j] * scale * (to_f32(w.v[j]) + a.offset), o.v[j]);
            store_vec<E, MODE, VEC>(out, c0, a.H, o);
        }
    }
}

// Eight elements as fp32, from memory's form and back, rounded.
__device__ __forceinline__ void to_floats(const uint4& p, float (&v)[8], __nv_bfloat16) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void to_floats(const uint4& p, float (&v)[8], __half) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}
__device__ __forceinline__ uint32_t round_two(float lo, float hi, __nv_bfloat16) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}
__device__ __forceinline__ uint32_t round_two(float lo, float hi, __half) {
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}
// A vector of the stream: as it lies in memory, and as fp32.
template <typename S>
struct Raw {
    uint4 v[sizeof(S) / 2];
};
template <typename S>
__device__ __forceinline__ Raw<S> load_raw(const S* at) {
    Raw<S> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(S) / 2); ++i) r.v[i] = reinterpret_cast<const uint4*>(at)[i];
    return r;
}
template <typename S>
__device__ __forceinline__ void to_floats(const Raw<S>& r, float (&v)[8]) {
    if constexpr (sizeof(S) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(r.v[i].x); v[4 * i + 1] = __uint_as_float(r.v[i].y);
            v[4 * i + 2] = __uint_as_float(r.v[i].z); v[4 * i + 3] = __uint_as_float(r.v[i].w);
        }
    } else {
        to_floats(r.v[0], v, S{});
    }
}
template <typename S>
__device__ __forceinline__ void store_rounded(S* at, const float (&v)[8]) {
    if constexpr (sizeof(S) == 4) {
        reinterpret_cast<float4*>(at)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(at)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(at) = make_uint4(round_two(v[0], v[1], S{}), round_two(v[2], v[3], S{}), round_two(v[4], v[5], S{}),
                                                   round_two(v[6], v[7], S{}));
    }
}

// Many long rows of up to 8192 elements, all on their boundaries: a CTA per row, V vectors to a thread.  What bounds it are the instructions beside
// the loads, of which each warp's sums are a large part: fewer warps to a row, as many rows to an SM as their registers allow
// (us, 32768 rows of 7168 / 4096 of 4096 with an fp32 stream: V 1 by two rows to an SM 382 / 32.4, V 2 by three 293 / 32.4, V 4 by
// four 269 / 36.4, by five 297 / 41; rows in pairs by CTAs that stay, the next ones brought ahead, 383 / 50).
template <typename E, typename S, int V>
__global__ void __launch_bounds__(V == 2 ? 512 : 256, V == 2 ? 3 : 4) sandwich_row_kernel(BlockNormArgs a) {
    __shared__ float part[2][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    const E* const y = static_cast<const E*>(a.y) + t * a.ldy;
    const S* const r = a.r ? static_cast<const S*>(a.r) + t * a.ldr : nullptr;
    const float mean = 1.f / (float)a.H;
    uint4 yv[V];
    Raw<S> rv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c0 = 8 * (threadIdx.x + i * blockDim.x);
        yv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (c0 < a.H) {
            yv[i] = *reinterpret_cast<const uint4*>(y + c0);
            if (r) rv[i] = load_raw(r + c0);
        }
    }
    float g = a.row_gate ? __ldcg(a.row_gate + t) : 1.f;
    if (a.sigmoid) g = 1.f / (1.f + __expf(-g));
    if (a.post) {
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[8];
            to_floats(yv[i], f, E{});
#pragma unroll
            for (int j = 0; j < 8; ++j) sq += f[j] * f[j];
        }
        g *= rsqrtf(row_sum<0>(sq, part[0], lane, warp) * mean + a.eps);
    }
    float s[V][8], sq = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c0 = 8 * (threadIdx.x + i * blockDim.x);
        if (c0 < a.H) {
            float f[8];
            to_floats(yv[i], s[i], E{});
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] *= g;
            if (a.post) {
                to_floats(*reinterpret_cast<const uint4*>(static_cast<const E*>(a.post) + c0), f, E{});
                if (a.offset != 0.f) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] += a.offset;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) s[i][j] *= f[j];
            }
            if (a.gate) {
                to_floats(*reinterpret_cast<const uint4*>(static_cast<const E*>(a.gate) + c0), f, E{});
#pragma unroll
                for (int j = 0; j < 8; ++j) s[i][j] *= f[j];
            }
            if (r) {
                to_floats(rv[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[i][j] += a.scale * f[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sq += s[i][j] * s[i][j];
            store_rounded(static_cast<S*>(a.sum) + t * a.lds + c0, s[i]);
        }
    }
    if (!a.out) return;
    const float scale = rsqrtf(row_sum<0>(sq, part[1], lane, warp) * mean + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c0 = 8 * (threadIdx.x + i * blockDim.x);
        if (c0 < a.H) {
            float f[8];
            to_floats(*reinterpret_cast<const uint4*>(static_cast<const E*>(a.w) + c0), f, E{});
            if (a.offset != 0.f) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += a.offset;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i][j] *= scale * f[j];
            store_rounded(static_cast<E*>(a.out) + t * a.ldo + c0, s[i]);
        }
    }
}

constexpr int kBlockNormWarps = 8;

template <typename E, typename S, int MODE, int VPT>
cudaError_t launch_row_per_cta(const BlockNormArgs& a, int nvec, cudaStream_t st) {
    const int threads = ((nvec + VPT - 1) / VPT + 31) / 32 * 32;
    return launch_pdl(sandwich_norm_kernel<E, S, MODE, VPT, 0>, dim3(a.T), dim3(threads), st, a);
}
template <typename E, typename S, int MODE, int VPT>
cudaError_t launch_row_per_warp(const BlockNormArgs& a, cudaStream_t st) {
    return launch_pdl(sandwich_norm_kernel<E, S, MODE, VPT, kBlockNormWarps>,
                      dim3((unsigned)(((int64_t)a.T + kBlockNormWarps - 1) / kBlockNormWarps)), dim3(32 * kBlockNormWarps), st, a);
}

template <typename E, typename S, int MODE>
cudaError_t launch_mode(const BlockNormArgs& a, cudaStream_t st) {
    const int nvec = MODE == ROWS_SINGLE ? a.H : (a.H + (MODE == ROWS_SHIFTED ? 7 : 0) + 7) / 8;
    // Many short rows: a warp per row.  Few: a CTA per row has more loads in flight.
    if (a.T >= 4 * kBlockNormWarps) {
        if (nvec <= 32) return launch_row_per_warp<E, S, MODE, 1>(a, st);
        if (nvec <= 64) return launch_row_per_warp<E, S, MODE, 2>(a, st);
        if (nvec <= 128) return launch_row_per_warp<E, S, MODE, 4>(a, st);
    }
    if constexpr (MODE == ROWS_ALIGNED) {
        const auto row = [&](auto kernel, int v) {
            return launch_pdl(kernel, dim3(a.T), dim3(((nvec + v - 1) / v + 31) / 32 * 32), st, a);
        };
        // sandwich_row_kernel from where its rows to an SM tell.  us, this kernel / V 2 / V 4, rows of
        //   16 bits    512 rows        1024 rows           4096 rows           16384 rows
        //     2048   3.9/4.3/5.4    5.8/6.0/6.3     15.2/13.8/15.6      50.3/43.5/44.7
        //     4096   6.0/6.2/6.5    9.8/9.6/8.7     28.7/25.3/25.5      99.0/82.1/82.6
        //     5120   8.0/6.3/7.3  12.1/10.9/12.8    36.9/32.4/32.0     128.9/107.2/102.1
        //     8192  10.7/10.2/8.7 17.7/15.2/16.1    58.5/47.2/46.2     212.4/164.8/158.4
        //   fp32 stream
        //     2048   4.6/5.3/6.5    6.5/7.5/7.9     18.6/19.8/22.0      61.1/62.0/68.3
        //     4096   7.2/7.7/8.7  12.0/13.0/12.0    34.9/34.6/39.9     122.0/118.4/127.4
        //     8192  13.2/13.5/12.2 21.9/21.3/23.1   71.8/64.2/69.3     264.6/230.3/244.1
        // (33 to 256 rows: this kernel by 5 to 25 %, 384 rows: within 20 % either way.)
        const bool rows = sizeof(S) == 2 ? a.T >= 1024 || (a.T >= 512 && nvec > 512) : a.T >= 1024 && nvec >= 512;
        if (rows && nvec <= 1024)
            return nvec > 512 && sizeof(S) == 2 ? row(sandwich_row_kernel<E, S, 4>, 4) : row(sandwich_row_kernel<E, S, 2>, 2);
    }
    if (nvec <= 1024) return launch_row_per_cta<E, S, MODE, 1>(a, nvec, st);
    if (nvec <= 2048 || MODE == ROWS_ALIGNED) return launch_row_per_cta<E, S, MODE, 2>(a, nvec, st);
    if constexpr (MODE == ROWS_SHIFTED) return launch_row_per_cta<E, S, MODE, 3>(a, nvec, st);
    if constexpr (MODE == ROWS_SINGLE) {
        if (nvec <= 4096) return launch_row_per_cta<E, S, MODE, 4>(a, nvec, st);
        if (nvec <= 8192) return launch_row_per_cta<E, S, MODE, 8>(a, nvec, st);
        return launch_row_per_cta<E, S, MODE, 16>(a, nvec, st);
    }
    return cudaErrorInvalidValue;
}

template <typename E, typename S>
cudaError_t launch_type(const BlockNormArgs& a, cudaStream_t st) {
    // how far each tensor's rows start off a boundary of 8 elements: `first` of row 0, and `pitch` more with
    // each row
    const bool many = a.T > 1;
    const int first = off_boundary<E>(a.y), pitch = many ? (int)(a.ldy & 7) : 0;
    const auto alike = [&](const void* p, int off, int64_t ld) {
        return !p || (off == first && (!many || (int)(ld & 7) == pitch));
    };
    // fp32 vectors move as two halves of 16 bytes
    if (!alike(a.r, off_boundary<S>(a.r), a.ldr) || !alike(a.sum, off_boundary<S>(a.sum), a.lds) ||
        !alike(a.out, off_boundary<E>(a.out), a.ldo))
        return launch_mode<E, S, ROWS_SINGLE>(a, st);
    const auto whole = [](const void* p) { return !p || off_boundary<E>(p) == 0; };
    if (first == 0 && pitch == 0 && a.H % 8 == 0 && whole(a.post) && whole(a.gate) && whole(a.w))
        return launch_mode<E, S, ROWS_ALIGNED>(a, st);
    return launch_mode<E, S, ROWS_SHIFTED>(a, st);
}

}  // namespace

cudaError_t launch_sandwich_norm(const moe_sandwich_desc& d, const void* x, const void* residual, const void* post_weight,
                                 const void* gate, const float* row_gate, const void* weight, void* sum_out, void* out,
                                 cudaStream_t st) {
    const BlockNormArgs a{x, residual, post_weight, gate, weight, row_gate, sum_out, out, d.ldx, d.ldr, d.lds, d.ldo,
                          d.T, d.H, d.row_sigmoid, d.eps, d.residual_scale, d.weight_offset};
    const bool f16 = d.dtype == MOE_DT_F16;
    if (d.wide) return f16 ? launch_type<__half, float>(a, st) : launch_type<__nv_bfloat16, float>(a, st);
    return f16 ? launch_type<__half, __half>(a, st) : launch_type<__nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace moe
