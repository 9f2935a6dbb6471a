// linear.cu -- y = f(x W^T + b) [* (x V^T + c)] [+ r], fp32 sums, one rounding.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float f, __nv_bfloat16& v) { v = __float2bfloat16_rn(f); }
__device__ __forceinline__ void from_f32(float f, __half& v) { v = __float2half_rn(f); }

__device__ __forceinline__ float apply_func(int func, float z) {
    switch (func) {
        case MOE_FUNC_SILU: return z / (1.f + __expf(-z));
        case MOE_FUNC_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678f));
        // 0.5 (1 + tanh u) = sigmoid(2 u)
        case MOE_FUNC_GELU_TANH: return z / (1.f + __expf(-1.5957691f * (z + 0.044715f * z * z * z)));
        case MOE_FUNC_RELU: return fmaxf(z, 0.f);
    }
    return z;
}

// 32 x 32 outputs per CTA of 256 threads, K in steps of 32 through shared memory.
template <typename E>
__global__ void __launch_bounds__(256)
linear_kernel(moe_linear_desc d, const E* x, const E* w, const E* w2, const float* b, const float* b2,
              const E* r, E* out) {
    __shared__ float xs[32][33], ws[32][33], vs[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int n0 = blockIdx.x * 32;
    for (int64_t t0 = (int64_t)blockIdx.y * 32; t0 < d.T; t0 += (int64_t)gridDim.y * 32) {
        float z[4] = {}, u[4] = {};
        for (int k0 = 0; k0 < d.K; k0 += 32) {
            for (int i = ty; i < 32; i += 8) {
                const bool kin = k0 + tx < d.K;
                xs[i][tx] = kin && t0 + i < d.T ? to_f32(x[(t0 + i) * d.ldx + k0 + tx]) : 0.f;
                ws[i][tx] = kin && n0 + i < d.N ? to_f32(w[(int64_t)(n0 + i) * d.ldw + k0 + tx]) : 0.f;
                vs[i][tx] = w2 && kin && n0 + i < d.N ? to_f32(w2[(int64_t)(n0 + i) * d.ldw + k0 + tx]) : 0.f;
            }
            __syncthreads();
            for (int k = 0; k < 32; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[i] += xs[ty + 8 * i][k] * ws[tx][k];
                    u[i] += xs[ty + 8 * i][k] * vs[tx][k];
                }
            __syncthreads();
        }
        const int n = n0 + tx;
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t0 + ty + 8 * i;
            if (t >= d.T || n >= d.N) continue;
            float y = apply_func(d.func, z[i] + (b ? b[n] : 0.f));
            if (w2) y *= u[i] + (b2 ? b2[n] : 0.f);
            if (r) y += to_f32(r[t * d.ldr + n]);
            from_f32(y, out[t * d.ldo + n]);
        }
    }
}

}  // namespace

cudaError_t launch_linear(const moe_linear_desc& d, const void* x, const void* w, const void* w_mul,
                          const float* bias, const float* bias_mul, const void* residual, void* out,
                          int32_t* status, cudaStream_t st) {
    (void)status;
    const int64_t rows = ((int64_t)d.T + 31) / 32;
    const dim3 grid((d.N + 31) / 32, (unsigned)(rows < 65535 ? rows : 65535));
    if (d.dtype == MOE_DT_F16)
        linear_kernel<__half><<<grid, 256, 0, st>>>(
            d, static_cast<const __half*>(x), static_cast<const __half*>(w), static_cast<const __half*>(w_mul),
            bias, bias_mul, static_cast<const __half*>(residual), static_cast<__half*>(out));
    else
        linear_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(
            d, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(w),
            static_cast<const __nv_bfloat16*>(w_mul), bias, bias_mul,
            static_cast<const __nv_bfloat16*>(residual), static_cast<__nv_bfloat16*>(out));
    return cudaGetLastError();
}

}  // namespace moe
