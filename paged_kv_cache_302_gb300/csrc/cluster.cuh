// cluster.cuh -- thread-block clusters: barrier, distributed shared memory, launch.
#pragma once

#include <atomic>

#include "pa_device.cuh"

namespace pa {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of the cluster's CTAs: writes before it are visible to the other CTAs after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same in two halves, neither of which orders memory: after the second every CTA of the cluster has started, so
// that its shared memory may be written.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// fp32 at shared-memory address `a` of the cluster's CTA `rank`.
__device__ __forceinline__ float ld_cluster(uint32_t a, int rank) {
    float v;
    asm volatile("{\n\t.reg .b32 t;\n\tmapa.shared::cluster.u32 t, %1, %2;\n\tld.shared::cluster.f32 %0, [t];\n\t}"
                 : "=f"(v)
                 : "r"(a), "r"(rank)
                 : "memory");
    return v;
}

// Address in the cluster's window of shared-memory address `a` of CTA `rank`, and a store there.
__device__ __forceinline__ uint32_t map_cluster(uint32_t a, int rank) {
    uint32_t t;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(t) : "r"(a), "r"(rank));
    return t;
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Host: as launch_kernel, in clusters of `size` CTAs.
template <typename... KArgs, typename... Args>
static cudaError_t launch_clusters(void (*kern)(KArgs...), int size, dim3 grid, dim3 block, size_t smem,
                                   cudaStream_t st, Args&&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Host: how many clusters of 1, 2, 4 or 8 CTAs of a kernel the current device holds at once (its SMs come in groups
// that a cluster does not cross, so that not all of them fill up).  Asked once per device and kernel.
class ClusterRoom {
public:
    template <typename... KArgs>
    cudaError_t get(void (*kern)(KArgs...), int size, int threads, size_t smem, int* clusters) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const int k = size == 8 ? 3 : size == 4 ? 2 : size == 2 ? 1 : 0;
        std::atomic<int>* slot = dev < kDevices ? &known_[dev][k] : nullptr;
        if (slot && (*clusters = slot->load(std::memory_order_relaxed)) > 0) return cudaSuccess;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)size);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(clusters, kern, &cfg);
        if (e == cudaSuccess && slot) slot->store(*clusters, std::memory_order_relaxed);
        return e;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> known_[kDevices][4] = {};
};

}  // namespace pa
