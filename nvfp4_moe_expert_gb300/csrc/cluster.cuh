// Thread-block clusters: rank, barrier, and another CTA's shared memory.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace nvfp4 {

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
// Every thread of the cluster; what they wrote to shared memory before is visible to all after.  In two parts, between which
// work goes on.  The warp's lanes come together first: the aligned forms take them to arrive as one, and branches of single
// lanes often stand in front.
__device__ __forceinline__ void cluster_barrier_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_barrier_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_barrier() {
    cluster_barrier_arrive();
    cluster_barrier_wait();
}
// Address of CTA `rank`'s copy of a shared-memory variable.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float cluster_load_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int cluster_load_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
// Arrive on another CTA's barrier (`addr`: cluster_addr of it): what this thread knows is done is visible to who waits there.
__device__ __forceinline__ void cluster_arrive(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Bounded wait on a barrier that CTAs of the cluster arrive on.
__device__ __forceinline__ bool cluster_wait_bounded(uint64_t* bar, uint32_t parity, const volatile int* abort, long long budget) {
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (abort != nullptr && *abort) return false;
        if (clock64() - t0 > budget) return false;
    }
}

}  // namespace nvfp4
