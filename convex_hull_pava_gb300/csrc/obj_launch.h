// Launches of the training objectives' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "iso_internal.h"

namespace isodev {

// A launch of clusters; `early`: it may start before the kernel in front of it in the stream has
// ended (the kernel waits where it needs that one's results).
struct ClusterLaunch {
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute at[2]{};
    ClusterLaunch(int64_t grid, int threads, size_t shared, int ctas, bool early, cudaStream_t st) {
        c.gridDim = dim3((unsigned)grid);
        c.blockDim = dim3(threads);
        c.dynamicSmemBytes = shared;
        c.stream = st;
        c.attrs = at;
        if (ctas > 1) {
            at[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
            at[c.numAttrs].val.clusterDim.x = ctas;
            at[c.numAttrs].val.clusterDim.y = at[c.numAttrs].val.clusterDim.z = 1;
            ++c.numAttrs;
        }
        if (early) {
            at[c.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[c.numAttrs].val.programmaticStreamSerializationAllowed = 1;
            ++c.numAttrs;
        }
    }
    ClusterLaunch(const ClusterLaunch&) = delete;
    template <class... P, class... A>
    cudaError_t operator()(void (*kernel)(P...), A... args) {
        const cudaError_t e = cudaLaunchKernelEx(&c, kernel, P(args)...);
        if (e != cudaSuccess) cudaGetLastError();  // reported here: not to a later call as well
        return e;
    }
};

// The clusters of `ctas` CTAs of a kernel that the GPU holds at once (a cluster's CTAs share a
// group of SMs, so that they are fewer than its SMs alone would take); asked once for each `held`
// (by several threads at first, if they call at once: they find the same).
using Held = std::atomic<int>[64][4];
template <class F>
cudaError_t clusters_held(F* kernel, const cudaLaunchConfig_t& config, int ctas, Held& held, int* fit) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::atomic<int>& known = held[dev][ctas == 1 ? 0 : ctas == 2 ? 1 : ctas == 4 ? 2 : 3];
    int n = known.load(std::memory_order_acquire);
    if (n == 0) {
        const int shared = (int)config.dynamicSmemBytes;
        if (shared > 48 * 1024 &&
            (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared)) != cudaSuccess)
            return e;
        if (ctas == 1) {
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, (int)config.blockDim.x, shared);
            n *= device_sms();
        } else {
            cudaLaunchConfig_t c = config;
            c.gridDim = dim3((unsigned)(device_sms() * ctas));
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &c);
        }
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
        n = std::max(1, n);
        known.store(n, std::memory_order_release);
    }
    *fit = n;
    return cudaSuccess;
}

template <class F>
cudaError_t by_type(int dtype, F f) {
    switch (dtype) {
        case ISO_F32: return f(float{});
        case ISO_BF16: return f(__nv_bfloat16{});
        default: return f(__half{});
    }
}

}  // namespace isodev
