// adapters.cu -- a dense layer with low-rank adapters of many requests:
// out = f(x W^T + b + v_w B_w^T) [* (x V^T + c + v_v B_v^T)] [+ r], v = scale x A^T, each row with its own adapter.
//
// Two launches: the low-rank products of every row (a warp each), and the layer, a thread per output.
#include "kernels.h"
#include "rows.cuh"

namespace moe {

namespace {

struct AdapterArgs {
    int T, N, K, R, L, func;
    int64_t ldx, ldw, ldr, ldo, lda, sa, ldb, sb;
    const void *x, *w[2], *a[2], *b[2], *res;
    const float *bias[2], *scale;
    const int32_t* ids;
    float* v[2];  // [T][R]
    void* out;
    int32_t* status;
};

__device__ __forceinline__ int adapter_of(const AdapterArgs& g, int64_t t) {
    const int j = __ldg(g.ids + t);
    return j >= 0 && j < g.L ? j : -1;
}

// grid (rows, matrices): a warp per low-rank product.
template <typename E>
__global__ void low_rank_kernel(AdapterArgs g) {
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int m = g.a[0] ? (int)blockIdx.y : 1, j = adapter_of(g, t);
    if (j < 0) {
        if (threadIdx.x == 0 && __ldg(g.ids + t) != -1) status_or(g.status, MOE_DEV_BAD_ADAPTER_ID);
        return;
    }
    const E* x = static_cast<const E*>(g.x) + t * g.ldx;
    for (int r = threadIdx.x / 32; r < g.R; r += blockDim.x / 32) {
        const E* a = static_cast<const E*>(g.a[m]) + j * g.sa + r * g.lda;
        float s = 0.f;
        for (int k = threadIdx.x % 32; k < g.K; k += 32) s += to_f32(x[k]) * to_f32(a[k]);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x % 32 == 0) g.v[m][t * g.R + r] = s * (g.scale ? __ldg(g.scale + j) : 1.f);
    }
}

template <typename E>
__global__ void layer_kernel(AdapterArgs g) {
    pdl_wait();
    const int64_t t = (int64_t)blockIdx.y * 16 + threadIdx.y;
    const int n = blockIdx.x * 16 + threadIdx.x;
    if (t >= g.T || n >= g.N) return;
    const int j = adapter_of(g, t);
    const E* x = static_cast<const E*>(g.x) + t * g.ldx;
    float z[2] = {0.f, 0.f};
    for (int m = 0; m < 2; ++m) {
        if (!g.w[m]) continue;
        const E* w = static_cast<const E*>(g.w[m]) + n * g.ldw;
        for (int k = 0; k < g.K; ++k) z[m] += to_f32(x[k]) * to_f32(w[k]);
        if (g.bias[m]) z[m] += g.bias[m][n];
        if (j < 0 || !g.b[m]) continue;
        const E* b = static_cast<const E*>(g.b[m]) + j * g.sb + n * g.ldb;
        for (int r = 0; r < g.R; ++r) z[m] += g.v[m][t * g.R + r] * to_f32(b[r]);
    }
    float y = z[0];
    switch (g.func) {
        case MOE_FUNC_SILU: y = y / (1.f + __expf(-y)); break;
        case MOE_FUNC_GELU: y = 0.5f * y * (1.f + erff(y * 0.70710678f)); break;
        case MOE_FUNC_GELU_TANH: y = y / (1.f + __expf(-1.5957691f * (y + 0.044715f * y * y * y))); break;
        case MOE_FUNC_RELU: y = y < 0.f ? 0.f : y; break;
    }
    if (g.w[1]) y *= z[1];
    if (g.res) y += to_f32(static_cast<const E*>(g.res)[t * g.ldr + n]);
    from_f32(y, static_cast<E*>(g.out)[t * g.ldo + n]);
}

template <typename E>
cudaError_t launch(const AdapterArgs& g, cudaStream_t st) {
    const cudaError_t err = launch_pdl(low_rank_kernel<E>, dim3(g.T, g.a[0] && g.a[1] ? 2 : 1), dim3(256), st, g);
    if (err != cudaSuccess) return err;
    return launch_pdl(layer_kernel<E>, dim3((g.N + 15) / 16, (g.T + 15) / 16), dim3(16, 16), st, g);
}

}  // namespace

cudaError_t launch_linear_adapters(const moe_linear_desc& d, const moe_adapter_desc& ad, const void* x, const void* w,
                                   const void* w_mul, const float* bias, const float* bias_mul, const void* residual,
                                   void* out, void* workspace, int32_t* status, cudaStream_t st) {
    const AdapterProducts p = AdapterProducts::plan(d.T, ad.R, ad.a && ad.a_mul ? 2 : 1);
    float* v0 = static_cast<float*>(workspace);
    float* v1 = ad.a ? v0 + p.plane / sizeof(float) : v0;
    const AdapterArgs g{d.T, d.N, d.K, ad.R, ad.L, d.func, d.ldx, d.ldw, d.ldr, d.ldo, ad.lda, ad.sa, ad.ldb, ad.sb,
                        x, {w, w_mul}, {ad.a, ad.a_mul}, {ad.b, ad.b_mul}, residual, {bias, bias_mul}, ad.scale, ad.ids,
                        {v0, v1}, out, status};
    return d.dtype == MOE_DT_F16 ? launch<__half>(g, st) : launch<__nv_bfloat16>(g, st);
}

}  // namespace moe
