// Layout and checks of the paged 4-bit cache (shared by its kernels).
#pragma once

#include <atomic>

#include <cuda_bf16.h>

#include "kvq_device.cuh"

namespace kvq {

constexpr int kGroup = 16;  // tokens per group of a page, and channels per scale

// Byte sizes inside the pool for head dimension D.
template <int D>
struct Paged {
    static constexpr int kRow = D / 2;                    // code bytes of a token's head
    static constexpr int kScales = D / kGroup;            // scale bytes of a token's head
    static constexpr int kHalf = kGroup * (kRow + kScales);  // keys (or values) of a group
    static constexpr int kBytes = 2 * kHalf;              // a group, keys then values
};
__host__ __device__ inline int paged_group_bytes(int D) { return 18 * D; }

// Bytes from the pool's start to group g of (page, kv head).
__device__ __forceinline__ size_t group_at(const kvq_paged_cfg& c, int page, int h, int g) {
    const int gpp = c.page_tokens / kGroup;
    return (((size_t)page * c.Hkv + h) * gpp + g) * (size_t)paged_group_bytes(c.D);
}

// Four code bytes to four fp16 pairs (low nibble in the low half); exact.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
// Two E4M3 bytes to an fp16 pair (low byte in the low half); exact.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Kernels of the paged cache are launched with leave to start before the one ahead in the stream
// has ended: after_previous waits until that has, and its writes are seen; before it nothing of
// the caller's memory is touched, and no thread returns.  let_next gives the same leave on.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// One 16-bit value of the cache's type, either way.
template <bool BF>
__device__ __forceinline__ float lo16(uint32_t w) {
    return BF ? __uint_as_float(w << 16) : __half2float(__ushort_as_half((uint16_t)w));
}
template <bool BF>
__device__ __forceinline__ float hi16(uint32_t w) {
    return BF ? __uint_as_float(w & 0xffff0000u) : __half2float(__ushort_as_half((uint16_t)(w >> 16)));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (BF) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    } else {
        return pack_h2(lo, hi);
    }
}

}  // namespace kvq

namespace kvq_host {
// A kernel's leave to use more shared memory than the default, asked for once per device.
struct SmemOptIn {
    std::atomic<uint64_t> done{0};
    int set(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t ce = cudaGetDevice(&dev);
        if (ce) return record_cuda(ce);
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (done.load(std::memory_order_relaxed) & bit) return KVQ_OK;
        ce = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (ce) return record_cuda(ce);
        done.fetch_or(bit, std::memory_order_relaxed);
        return KVQ_OK;
    }
};
// Launch in clusters of `cluster` blocks, overlapping the start with the kernel ahead.
template <typename... P, typename... A>
int launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                      A... args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    return record_cuda(cudaLaunchKernelEx(&lc, kernel, static_cast<P>(args)...));
}
int check_paged_cfg(const kvq_paged_cfg* cfg);
int check_paged_cache(const kvq_paged_cache* cache);
}  // namespace kvq_host
