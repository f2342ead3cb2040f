// Host side of kernels launched in clusters or as persistent grids, shared by
// the 8-bit products and the orthogonalisation: one-time set-up of a kernel on a
// device, and its launch.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "device.h"
#include "launch.h"

namespace tmmo {

// How many clusters of a kernel can run at a time, for every device: 0 until
// it is asked for, -1 where none fits.
struct ClusterCaps {
    std::mutex mu;
    int cap[kMaxDevices] = {};
};

// A launch of `blocks` blocks in clusters of `size`; dependent: a programmatic
// dependent of the launch before it.
struct ClusterLaunch {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];

    ClusterLaunch(unsigned blocks, int size, int threads, int smem, cudaStream_t stream,
                  bool dependent = false)
    {
        unsigned n = 0;
        if (dependent) {
            attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[n++].val.programmaticStreamSerializationAllowed = 1;
        }
        if (size > 1) {
            attr[n].id = cudaLaunchAttributeClusterDimension;
            attr[n].val.clusterDim.x = static_cast<unsigned>(size);
            attr[n].val.clusterDim.y = 1;
            attr[n++].val.clusterDim.z = 1;
        }
        cfg.gridDim = dim3(blocks, 1, 1);
        cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = n;
    }
    ClusterLaunch(const ClusterLaunch&) = delete;

    template <typename Kernel, typename... Args>
    cudaError_t run(Kernel kern, const Args&... args)
    {
        note_launch();
        const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, args...);
        return err != cudaSuccess ? err : cudaGetLastError();
    }
};

// Sets the kernel up on the current device (once) and gives the number of
// clusters of `size` blocks that fit it at a time; single blocks are not
// counted: one an SM.
template <typename Kernel>
cudaError_t cluster_cap(Kernel kern, ClusterCaps& caps, int size, int threads, int smem, int num_sms,
                        int* cap)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(caps.mu);
    if (caps.cap[dev] == 0) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err == cudaSuccess && size > 8)
            err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        int clusters = num_sms;
        if (err == cudaSuccess && size > 1) {
            ClusterLaunch l(static_cast<unsigned>(size * std::max(1, num_sms / size)), size, threads, smem,
                            nullptr);
            err = cudaOccupancyMaxActiveClusters(&clusters, kern, &l.cfg);
        }
        if (err != cudaSuccess)
            return err;
        caps.cap[dev] = clusters > 0 ? clusters : -1;
    }
    *cap = caps.cap[dev];
    return cudaSuccess;
}

}  // namespace tmmo
