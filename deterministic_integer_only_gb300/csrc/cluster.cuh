// Thread-block clusters: barrier and accesses to another CTA's shared
// memory. A launch without a cluster is one of a single CTA.
#pragma once
#include <stdint.h>

#include "int_device.cuh"
#include "ptx.cuh"

namespace detint {

__device__ __forceinline__ void cl_sync() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cl_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cl_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t cl_addr(const void* p, unsigned rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ int cl_ld32(const int* p, unsigned rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cl_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ i64 cl_ld64(const i64* p, unsigned rank) {
    i64 v;
    asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(cl_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ unsigned cl_ld32u(const unsigned* p, unsigned rank) { return (unsigned)cl_ld32((const int*)p, rank); }
__device__ __forceinline__ void cl_st64(u64* p, unsigned rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cl_addr(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void cl_st32(int* p, unsigned rank, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cl_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned cl_add32(unsigned* p, unsigned rank, unsigned v) {
    unsigned old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(cl_addr(p, rank)), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void cl_red32(unsigned* p, unsigned rank, unsigned v) {
    asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(cl_addr(p, rank)), "r"(v) : "memory");
}

}  // namespace detint
