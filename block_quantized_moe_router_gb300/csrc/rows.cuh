// rows.cuh -- rows of 16-bit or fp32 elements in vectors of 8, also where rows start off a vector's boundary
// (internal; the norms).
//
// Where rows start off a boundary of 8 elements, but all tensors' rows equally far off (an odd H, all
// contiguous), the vectors are laid over the row from the boundary before it: whole ones move as vectors, the
// two at the ends element by element, and a weight, which does not shift with the row, as two vectors shifted
// into one.  Where they are not equally far off, a vector is one element.
#pragma once
#include "common.cuh"

namespace moe {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float f, __nv_bfloat16& v) { v = __float2bfloat16_rn(f); }
__device__ __forceinline__ void from_f32(float f, __half& v) { v = __float2half_rn(f); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(float f, float& v) { v = f; }

enum { ROWS_ALIGNED, ROWS_SHIFTED, ROWS_SINGLE };

template <typename E, int VEC>
struct alignas(sizeof(E) * VEC < 16 ? sizeof(E) * VEC : 16) Pack {
    E v[VEC];
};

// VEC elements from column c0 on, those inside [0, H).
template <typename E, int MODE, int VEC>
__device__ __forceinline__ Pack<E, VEC> load_vec(const E* row, int c0, int H) {
    Pack<E, VEC> p;
    if (MODE != ROWS_SHIFTED || (c0 >= 0 && c0 + VEC <= H)) {
        p = *reinterpret_cast<const Pack<E, VEC>*>(row + c0);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            from_f32(0.f, p.v[j]);
            if (c0 + j >= 0 && c0 + j < H) p.v[j] = row[c0 + j];
        }
    }
    return p;
}
template <typename E, int MODE, int VEC>
__device__ __forceinline__ void store_vec(E* row, int c0, int H, const Pack<E, VEC>& p) {
    if (MODE != ROWS_SHIFTED || (c0 >= 0 && c0 + VEC <= H)) {
        *reinterpret_cast<Pack<E, VEC>*>(row + c0) = p;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (c0 + j >= 0 && c0 + j < H) row[c0 + j] = p.v[j];
    }
}

// Elements w[c0 .. c0 + 7], clamped to [0, H), where c0 may be off a 16-byte boundary: two aligned
// vectors shifted into one, or element by element where those reach beyond w.
template <typename E>
__device__ __forceinline__ Pack<E, 8> load_weight(const E* w, int c0, int H) {
    const int ow = (int)((reinterpret_cast<uintptr_t>(w) >> 1) & 7);
    const int shift = (c0 + ow) & 7, b0 = c0 - shift;  // w + b0 is aligned
    Pack<E, 8> p;
    if (b0 >= 0 && b0 + 16 <= H) {
        const uint4 lo = *reinterpret_cast<const uint4*>(w + b0), hi = *reinterpret_cast<const uint4*>(w + b0 + 8);
        uint32_t q[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 6; ++i) q[i] = shift & 4 ? q[i + 2] : q[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) q[i] = shift & 2 ? q[i + 1] : q[i];
        uint4 r;
        uint32_t* rw = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) rw[i] = shift & 1 ? __funnelshift_r(q[i], q[i + 1], 16) : q[i];
        p = *reinterpret_cast<Pack<E, 8>*>(&r);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p.v[j] = w[min(max(c0 + j, 0), H - 1)];
    }
    return p;
}

// Elements between a boundary of 8 elements and p.
template <typename E>
inline int off_boundary(const void* p) { return (int)((reinterpret_cast<uintptr_t>(p) / sizeof(E)) & 7); }

}  // namespace moe
