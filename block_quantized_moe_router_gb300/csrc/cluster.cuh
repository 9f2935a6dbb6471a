// cluster.cuh -- thread-block clusters: ranks, barriers, distributed shared memory, and the tensor
// maps of 16-bit matrices (internal).
#pragma once
#include <cudaTypedefs.h>
#include <stdint.h>

#include <atomic>

namespace moe {

// Lets `kernel` use `smem` bytes of dynamic shared memory (its largest need, so that no two calls differ)
// and clusters of up to 16; once per device.
template <typename K>
inline cudaError_t allow_large_launch(K* kernel, int smem, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err == cudaSuccess) err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return err;
}

// The warp's index, known to the compiler as one value for the warp.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }
// One lane of a converged warp.  Unlike a comparison with a lane number it tells the compiler that what
// follows runs on one thread, so that TMA and MMA operands need no search for a common value
// (4 % of moe_linear with few rows).
__device__ __forceinline__ bool elect_one() {
    __syncwarp();
    uint32_t p;
    asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// The cluster's barrier, for every thread of every CTA: shared-memory writes before the arrival are
// seen after the wait.  Arrivals and waits alternate.
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// The address of this CTA's shared-memory location `saddr` in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
__device__ __forceinline__ void st_cluster_v4(uint32_t mapped, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(mapped), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t mapped_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapped_bar) : "memory");
}

// Bounded wait on a phase of an mbarrier; false after kWaitNs.  One poll, and only where it finds nothing a
// loop with a clock: the loops that feed the tensor cores run on one thread, where every instruction
// between two waits counts (a counted loop and a look at a flag doubled the cost of a wait that has nothing
// to wait for).  The bound is a time and not a number of polls: a poll lasts up to 1 ms on a lone lane and
// 4 us on a whole warp.  All of it is in place: no call is made where one lane of a warp runs.
constexpr uint32_t kWaitHint = 1000000;  // ns that a poll may last
constexpr uint64_t kWaitNs = 4000000000ull;
__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ bool mbar_wait_suspended(uint64_t* bar, uint32_t parity) {
    const uint32_t addr = static_cast<uint32_t>(__cvta_generic_to_shared(bar));
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    if (__builtin_expect(ok != 0, 1)) return true;
    const uint64_t began = global_ns();
    do {
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(addr), "r"(parity), "r"(kWaitHint)
            : "memory");
    } while (ok == 0 && global_ns() - began < kWaitNs);
    return ok != 0;
}

// Place in a ring of stages: the slot, and the parity of its phase.  Counted, not divided: a division by
// a runtime number of stages took longer (600 cycles on a lone thread) than a stage's copies.
struct RingPos {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++slot == stages) {
            slot = 0;
            parity ^= 1u;
        }
    }
    __device__ __forceinline__ void back(int stages) {
        if (--slot < 0) {
            slot = stages - 1;
            parity ^= 1u;
        }
    }
};

// Tensor map of [rows][cols] 16-bit elements, rows ld apart: boxes of box_cols columns (64 or 32: 128
// or 64 bytes, swizzled over as many) x box_rows rows; what lies beyond reads as zero.
inline bool encode_rows16(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows,
                          int box_cols) {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
