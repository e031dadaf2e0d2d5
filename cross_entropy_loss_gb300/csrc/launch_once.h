// What a launch asks the runtime once for a kernel and device, kept in fixed arrays (nothing on the way to a
// launch allocates or throws).  Two threads that ask at once get the same answer.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "internal.h"

namespace foak {

constexpr int kMaxDevices = 64;

inline cudaError_t current_device(int* dev) {
    const cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return e;
    return *dev >= 0 && *dev < kMaxDevices ? cudaSuccess : cudaErrorInvalidDevice;
}

// Dynamic shared memory above 48 KB for one kernel.
struct SmemOnce {
    std::atomic<bool> done[kMaxDevices] = {};

    template <typename K>
    cudaError_t allow(K kernel, int bytes) {
        int dev = 0;
        cudaError_t e = current_device(&dev);
        if (e != cudaSuccess || done[dev].load(std::memory_order_acquire)) return e;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
        return e;
    }
};

// Clusters of one kernel that are resident at once, by cluster size (1, 2, 4, 8) and threads (32 .. 1024); the
// caller's shared memory goes by those two.
struct ResidentOnce {
    std::atomic<int> known[kMaxDevices][4][32] = {};

    template <typename K>
    cudaError_t count(K kernel, int cluster, int threads, size_t smem, int* clusters) {
        int dev = 0;
        cudaError_t e = current_device(&dev);
        if (e != cudaSuccess) return e;
        const int c = cluster == 1 ? 0 : cluster == 2 ? 1 : cluster == 4 ? 2 : 3;
        std::atomic<int>& at = known[dev][c][threads / 32 - 1];
        *clusters = at.load(std::memory_order_relaxed);
        if (*clusters) return cudaSuccess;
        int n = 0;
        if (cluster == 1) {
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
            n *= device_sm_count();
        } else {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(cluster));
            cfg.blockDim = dim3(static_cast<unsigned>(threads));
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = static_cast<unsigned>(cluster);
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        }
        if (e != cudaSuccess) return e;
        at.store(*clusters = n > 0 ? n : 1, std::memory_order_relaxed);
        return cudaSuccess;
    }
};

}  // namespace foak
