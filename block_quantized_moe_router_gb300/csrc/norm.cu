// norm.cu -- residual add and RMS norm: s = x + r, y = s * rsqrt(mean(s^2) + eps) * weight.
//
// One CTA per row.  The row stays in registers between the sum of squares and the scaling, so
// every input is read once and every output written once; the kernel is bound by HBM.  The sum
// s, its squares and the scaling are fp32; s and y are each rounded once, y from the unrounded s.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

// VEC elements of 2 bytes <-> fp32
template <typename E, int VEC>
struct alignas(2 * VEC) Pack {
    E v[VEC];
};
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float f, __nv_bfloat16& v) { v = __float2bfloat16_rn(f); }
__device__ __forceinline__ void from_f32(float f, __half& v) { v = __float2half_rn(f); }

struct NormArgs {
    const void *x, *r, *w;
    void *sum, *out;
    int64_t ldx, ldr, lds, ldo;
    int H;
    float eps;
};

template <typename E, int VEC, int VPT>
__global__ void __launch_bounds__(1024)
add_rms_norm_kernel(NormArgs a) {
    using P = Pack<E, VEC>;
    __shared__ float part[32];
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x;
    const int nvec = a.H / VEC, tid = threadIdx.x;
    const P* x = reinterpret_cast<const P*>(static_cast<const E*>(a.x) + row * a.ldx);
    const P* r = a.r ? reinterpret_cast<const P*>(static_cast<const E*>(a.r) + row * a.ldr) : nullptr;
    const P* w = reinterpret_cast<const P*>(a.w);
    P* sum = a.sum ? reinterpret_cast<P*>(static_cast<E*>(a.sum) + row * a.lds) : nullptr;
    P* out = reinterpret_cast<P*>(static_cast<E*>(a.out) + row * a.ldo);
    P xv[VPT], rv[VPT], wv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {  // every load issued before any is used
        const int c = tid + i * blockDim.x;
        if (c < nvec) {
            xv[i] = x[c];
            if (r) rv[i] = r[c];
            wv[i] = w[c];
        }
    }
    float s[VPT][VEC], sq = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * blockDim.x;
        if (c < nvec) {
            P o;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                s[i][j] = to_f32(xv[i].v[j]);
                if (r) s[i][j] += to_f32(rv[i].v[j]);
                sq += s[i][j] * s[i][j];
                from_f32(s[i][j], o.v[j]);
            }
            if (sum) sum[c] = o;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if ((tid & 31) == 0) part[tid >> 5] = sq;
    __syncthreads();
    sq = (tid & 31) < (blockDim.x >> 5) ? part[tid & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    const float scale = rsqrtf(sq / (float)a.H + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * blockDim.x;
        if (c < nvec) {
            P o;
#pragma unroll
            for (int j = 0; j < VEC; ++j) from_f32(s[i][j] * scale * to_f32(wv[i].v[j]), o.v[j]);
            out[c] = o;
        }
    }
}

template <typename E, int VEC, int VPT>
cudaError_t launch_vpt(const NormArgs& a, int T, int threads, cudaStream_t st) {
    return launch_pdl(add_rms_norm_kernel<E, VEC, VPT>, dim3(T), dim3(threads), st, a);
}

template <typename E, int VEC>
cudaError_t launch_vec(const NormArgs& a, int T, cudaStream_t st) {
    const int nvec = a.H / VEC;
    int vpt = 1;
    while (vpt * 1024 < nvec) vpt *= 2;
    const int threads = ((nvec + vpt - 1) / vpt + 31) / 32 * 32;
    switch (vpt) {
        case 1: return launch_vpt<E, VEC, 1>(a, T, threads, st);
        case 2: return launch_vpt<E, VEC, 2>(a, T, threads, st);
    }
    if constexpr (VEC < 8) {
        switch (vpt) {
            case 4: return launch_vpt<E, VEC, 4>(a, T, threads, st);
            case 8: return launch_vpt<E, VEC, 8>(a, T, threads, st);
        }
        if constexpr (VEC < 2) {
            if (vpt == 16) return launch_vpt<E, VEC, 16>(a, T, threads, st);
        }
    }
    return cudaErrorInvalidValue;
}

template <typename E>
cudaError_t launch_type(const NormArgs& a, int T, cudaStream_t st) {
    // The widest vector that every row's start and the row length allow.
    uint64_t bits = (uint64_t)a.H | (uint64_t)(uintptr_t)a.x / 2 | (uint64_t)(uintptr_t)a.w / 2 |
                    (uint64_t)(uintptr_t)a.out / 2;
    if (T > 1) bits |= (uint64_t)a.ldx | (uint64_t)a.ldo;
    if (a.r) bits |= (uint64_t)(uintptr_t)a.r / 2 | (T > 1 ? (uint64_t)a.ldr : 0);
    if (a.sum) bits |= (uint64_t)(uintptr_t)a.sum / 2 | (T > 1 ? (uint64_t)a.lds : 0);
    if (bits % 8 == 0) return launch_vec<E, 8>(a, T, st);
    if (bits % 2 == 0) return launch_vec<E, 2>(a, T, st);
    return launch_vec<E, 1>(a, T, st);
}

}  // namespace

cudaError_t launch_add_rms_norm(const moe_norm_desc& d, const void* x, const void* r, const void* w,
                                void* sum, void* out, cudaStream_t st) {
    const NormArgs a{x, r, w, sum, out, d.ldx, d.ldr, d.lds, d.ldo, d.H, d.eps};
    return d.dtype == MOE_DT_F16 ? launch_type<__half>(a, d.T, st)
                                 : launch_type<__nv_bfloat16>(a, d.T, st);
}

}  // namespace moe
