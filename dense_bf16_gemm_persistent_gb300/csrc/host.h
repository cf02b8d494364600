// Host-side services that the library's translation units share: the calling thread's
// error message, the device's properties and the description of the last plan.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "../../include/gbgemm.h"

namespace gb {
namespace host {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

// Empty the calling thread's error message (at the start of an entry point).
void clear_error();

// Record a message for gb_last_error() and return `s`.
gb_status_t fail(gb_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gb_status_t cuda_fail(cudaError_t e, const char* what);

struct DeviceInfo {
    bool ready = false;
    int sms = 0;
    int major = 0, minor = 0;
    size_t smem_optin = 0;
};

// The current device's ordinal and properties (read once); refuses a device that is not sm_103.
gb_status_t device_info(int* dev_out, DeviceInfo* info);

// The plan of the 4-bit products as gb_set_config() fixes it; 0: not.
struct W4Override {
    int cluster, k_warps;
};
W4Override w4_override();

// What gb_last_plan() reports: a static format that takes six %lld.
void note_plan(const char* fmt, long long a, long long b, long long c, long long d, long long e, long long f);
// The same of a call that had nothing to do.
void note_empty();

// A launch whose CTAs may be set up while the kernel before it in the stream still runs: the kernel
// must wait (ptx.cuh: wait_for_earlier_kernels) before it touches global memory.
struct Launch {
    cudaLaunchConfig_t config = {};
    cudaLaunchAttribute attributes[2];

    Launch(dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster = 1) {
        config.gridDim = grid;
        config.blockDim = block;
        config.dynamicSmemBytes = smem;
        config.stream = stream;
        config.attrs = attributes;
        config.numAttrs = cluster > 1 ? 2 : 1;
        attributes[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attributes[0].val.programmaticStreamSerializationAllowed = 1;
        attributes[1].id = cudaLaunchAttributeClusterDimension;
        attributes[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attributes[1].val.clusterDim.y = 1;
        attributes[1].val.clusterDim.z = 1;
    }

    template <class Kernel, class... Args>
    gb_status_t operator()(const char* what, Kernel kernel, Args... args) {
        const cudaError_t e = cudaLaunchKernelEx(&config, kernel, args...);
        return e == cudaSuccess ? GB_OK : cuda_fail(e, what);
    }
};

// More than the default 48 KB of dynamic shared memory, once for each kernel and device.  (Two
// threads may both set the attribute: to the same value.)
template <class Kernel>
gb_status_t allow_smem(Kernel kernel, std::atomic<bool>* ready, int dev, size_t most) {
    if (ready[dev].load(std::memory_order_acquire)) return GB_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    ready[dev].store(true, std::memory_order_release);
    return GB_OK;
}

// Clusters of a size that run at once (a GPC's SMs hold whole clusters only: of blocks that fit two on each of 152 SMs, 36
// clusters of eight), asked for once for each kernel, device and size.
struct ClusterCounts {
    std::atomic<int> known[64][9] = {};

    template <class Kernel>
    gb_status_t get(Kernel kernel, int threads, size_t smem, int dev, int cluster, int64_t* count) {
        int n = known[dev][cluster].load(std::memory_order_relaxed);
        if (n == 0) {
            Launch launch(cluster, threads, smem, nullptr, cluster);
            launch.config.numAttrs = 2;  // (a cluster of one too)
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &launch.config);
            if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
            known[dev][cluster].store(n, std::memory_order_relaxed);
        }
        *count = n;
        return GB_OK;
    }
};

inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace host
}  // namespace gb
