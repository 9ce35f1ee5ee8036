// Thread-block clusters: barriers, words sent to another CTA, launch.
#pragma once

#include "common.cuh"

namespace dfl {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Arrival at a barrier of the cluster that orders no memory but what a fence before
// it does (fence_mbar_init for mbarriers), so that no store in flight is waited for.
// A warp whose lanes come from different branches arrives as one.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}

// Orders this thread's memory accesses, and those it has seen ordered before them, with
// the cluster's, for an arrival that orders none.
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

// Sends a word to where p lies in this CTA, in CTA `rank`, and four bytes to its
// mbarrier that lies where bar does.
__device__ __forceinline__ void send_word(void* p, uint64_t* bar, uint32_t rank, uint32_t v) {
    uint32_t at, b;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(at), "r"(v), "r"(b)
                 : "memory");
}

// launch_k with clusters of `ranks` CTAs in a row.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_cluster_k(void (*kern)(KArgs...), dim3 grid, dim3 block, int ranks, cudaStream_t s, size_t smem,
                                    Args&&... args) {
    set_carveout_once(reinterpret_cast<const void*>(kern));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = g_pdl ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    ++g_launches;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace dfl
