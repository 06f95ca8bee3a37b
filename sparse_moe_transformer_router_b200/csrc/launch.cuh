// launch.cuh -- host helpers the library's launches share: programmatic
// stream serialisation, the kernels' shared-memory limits, and the error
// message of entry points that take no handle.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <utility>

#include "l4moe.h"

namespace l4moe {

// Whether a bytes at p and b bytes at q share any.
inline bool overlap(const void* p, size_t a, const void* q, size_t b) {
    const uintptr_t u = reinterpret_cast<uintptr_t>(p), v = reinterpret_cast<uintptr_t>(q);
    return u < v + b && v < u + a;
}

// Record msg for l4moe_last_error(NULL) (this thread's) and return s.
l4moe_status op_fail(l4moe_status s, const char* msg) noexcept;

// Every kernel goes out with programmatic stream serialisation: it may begin
// launching while the previous kernel of the stream finishes, and waits for
// it (pdl_enter) before touching memory, which hides the launch gaps of the
// short kernels of a small batch.  Launch errors are left for
// cudaGetLastError, like a <<<>>> launch.
// cluster.x > 0 also launches the grid as clusters of that shape.
template <typename... KArgs, typename... Args>
void launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                    const unsigned (&cluster)[3], Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cluster[0] > 0) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster[0];
        attr[1].val.clusterDim.y = cluster[1];
        attr[1].val.clusterDim.z = cluster[2];
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Clusters of (1, 1, cluster_z), or of (cluster_x, 1, 1); 0: none.
template <typename... KArgs, typename... Args>
void launch_kc(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
               unsigned cluster_z, Args&&... args) {
    const unsigned c[3] = {cluster_z > 0 ? 1u : 0u, 1u, cluster_z};
    launch_cluster(kernel, grid, block, smem, st, c, std::forward<Args>(args)...);
}
template <typename... KArgs, typename... Args>
void launch_cluster_x(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                      unsigned cluster_x, Args&&... args) {
    const unsigned c[3] = {cluster_x, 1u, 1u};
    launch_cluster(kernel, grid, block, smem, st, c, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
void launch_k(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
              Args&&... args) {
    launch_kc(kernel, grid, block, smem, st, 0u, std::forward<Args>(args)...);
}

template <typename K>
void set_smem_attr(K kernel, size_t bytes) {
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Raise a kernel's dynamic shared-memory limit once per device: the
// attribute belongs to the kernel's instance in each device's context, so a
// process that runs layers on several GPUs sets it on each.  `done` holds
// one bit per device index (devices 64 and up set it on every call).
template <typename K>
void ensure_smem_attr(std::atomic<uint64_t>& done, K kernel, size_t bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        set_smem_attr(kernel, bytes);
        return;
    }
    const uint64_t bit = 1ull << dev;
    if (done.load(std::memory_order_acquire) & bit) return;
    set_smem_attr(kernel, bytes);
    done.fetch_or(bit, std::memory_order_acq_rel);
}

}  // namespace l4moe
