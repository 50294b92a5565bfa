// launch.cuh -- kernel launches with programmatic dependent launch.
//
// A kernel launched here may start its CTAs while the previous kernel in the stream is
// still running (CUDA's programmatic stream serialisation). Every kernel launched this way
// calls griddep_wait() (common.cuh) in every CTA, which blocks until the previous grid has
// completed and its writes are visible; its own setup (barrier initialisation, tensor-memory
// allocation, tensor-map prefetch) runs before that and overlaps the previous kernel's last CTAs.
// Because each such kernel waits for its predecessor before it can complete, the ordering is
// transitive along the stream.
// In front of the wait a kernel writes no global memory and uses none that it reads, with two exceptions, both in paged
// attention:
//  - attention_paged_rows.cu and attention_paged_tc.cu prefetch to L2 there, by lengths and page entries that may still change:
//    bounds are checked, nothing of it is used, and all is read again behind the wait.
//  - attention_paged_rows.cu behind a prefix reads lengths, tables, queries and own keys before it waits. The grid in front of it
//    is the prefix's, of the same call, which writes scratch alone and lets dependents start only behind its own wait: what those
//    reads need was complete by then. Its wait, for the prefix's parts, stands before its first store.
// A kernel that lets dependents start (griddep_launch_dependents) does so behind its own wait.
// VIT_PDL=0 launches without the attribute (plain stream order).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <utility>

namespace vit {

inline bool pdl_enabled() {
    static const bool on = [] {
        const char* e = std::getenv("VIT_PDL");
        return !(e && e[0] == '0');
    }();
    return on;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                             Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The same in clusters of `cluster` CTAs along x (grid.x a multiple of it).
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, int cluster, size_t smem,
                                     cudaStream_t s, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// A kernel's dynamic shared-memory limit (cudaFuncSetAttribute) is set per device: raise
// it once on each device the kernel runs on. `done` holds one bit per device ordinal below
// 64 (others are set on every call).
template <typename... KArgs>
cudaError_t set_smem_limit_once(void (*kernel)(KArgs...), int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

}  // namespace vit
