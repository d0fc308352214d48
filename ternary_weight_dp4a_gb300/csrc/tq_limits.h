// tq_limits.h -- what the host has to know of a kernel before it launches it: its limit of dynamic shared
// memory, and how many of its clusters run at once.  Host code only.
#pragma once

#include <cuda_runtime.h>

#include <mutex>

namespace tq {

// A kernel's limit of dynamic shared memory.  The limit belongs to the function on a device, not
// to a launch: each kernel's is raised once per device, under a lock, to the most that any
// call can ask for, so that no thread's call lowers it under another's launch.
struct SmemLimit {
    static constexpr int kMaxDev = 64;
    std::mutex mu;
    bool raised[kMaxDev] = {};

    template <typename Kernel>
    cudaError_t raise(Kernel *kernel, size_t most) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lock(mu);
        if (dev < kMaxDev && raised[dev]) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
        if (e == cudaSuccess && dev < kMaxDev) raised[dev] = true;
        return e;
    }
};

// How many clusters of a kernel can run at once, asked for once per device and cluster size: a cluster's CTAs
// are SMs of one GPC, so it is fewer than the SMs divided by the size (2 x 76 SMs: 72 of two, 48 of three).
struct ClusterLimit {
    static constexpr int kMaxDev = 64, kMaxSize = 8;
    std::mutex mu;
    int known[kMaxDev][kMaxSize + 1] = {};

    template <typename Kernel>
    cudaError_t most(Kernel *kernel, int dev, int size, int threads, size_t smem, int sms, int *out) {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < kMaxDev && known[dev][size] > 0) {
            *out = known[dev][size];
            return cudaSuccess;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(sms / size * size));
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = static_cast<unsigned>(size);
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) return e;
        *out = n > 0 ? n : 1;
        if (dev < kMaxDev) known[dev][size] = *out;
        return cudaSuccess;
    }
};

}  // namespace tq
