// Thread-block clusters: a block's place in its cluster, the cluster barrier, reads of another
// block's shared memory, and launches over clusters.
#pragma once

#include "common.cuh"
#include "mbarrier.cuh"

namespace liger {

__device__ __forceinline__ uint32_t block_in_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t blocks_in_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// every thread of every block of the cluster; the warps converged
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// address of the same shared object in block `rank` of the cluster
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
    uint32_t o;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(o) : "r"(smem_u32(p)), "r"(rank) : "memory");
    return o;
}
__device__ __forceinline__ float peer_float(const float* p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float4 peer_float4(const float* p, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(peer(p, rank))
                 : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long peer_key(const unsigned long long* p, uint32_t rank) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void peer_store(int* p, uint32_t rank, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer(p, rank)), "r"(v) : "memory");
}

// launch_early over clusters of `cluster` blocks (gridDim a multiple of it in each dimension)
template <typename... P, typename... A>
int launch_cluster(const char* what, void (*kernel)(P...), dim3 grid, dim3 cluster, int threads, size_t smem, cudaStream_t st,
                   A... args) {
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster.x;
    at[1].val.clusterDim.y = cluster.y;
    at[1].val.clusterDim.z = cluster.z;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(static_cast<unsigned>(threads));
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = at;
    c.numAttrs = 2;
    cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
    return check_launch(what);
}

}  // namespace liger
