// Helpers of the kernel launchers: facts about the current device that every launch asks for,
// kept per device, and launches that overlap with their predecessor's end.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace harts {

constexpr int kMaxDeviceIds = 64;

inline int current_device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 ? dev : 0;
}

// SMs of the current device (152, a GB300's, where there is none: sizes can be asked for
// without a GPU).
inline int sm_count() {
    static std::atomic<int> known[kMaxDeviceIds];
    const int dev = current_device();
    if (dev < kMaxDeviceIds) {
        const int n = known[dev].load(std::memory_order_relaxed);
        if (n > 0) return n;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    if (dev < kMaxDeviceIds) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Allows `kernel` its dynamic shared memory, once per device.  `done` belongs to the kernel.
template <typename F>
inline cudaError_t allow_smem(F *kernel, int bytes, std::atomic<uint64_t> &done) {
    const int dev = current_device();
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// The library's own error word on the current device, for calls that are given none
// (harts_device_error reads it); nullptr where it cannot be had.
int32_t *own_error_word();

// The kernels of one call overlap at their seams: each allows the next one to be set up as
// soon as it runs itself, and waits for its predecessor only where it first needs (or
// overwrites) something of it.  The first kernel of a call is launched without this, so what
// came before the call is complete for all of them.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// `behind`: the kernel may be set up before its predecessor in the stream has ended (it waits
// itself, see wait_previous).
template <typename F, typename... P>
inline cudaError_t launch(F *kernel, int64_t blocks, int threads, size_t smem, int cluster, bool behind, cudaStream_t st,
                          const P &...p) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    cfg.attrs = at;
    cfg.numAttrs = 0;
    if (cluster > 1) {
        cudaLaunchAttribute &c = at[cfg.numAttrs++];
        c.id = cudaLaunchAttributeClusterDimension;
        c.val.clusterDim.x = cluster;
        c.val.clusterDim.y = c.val.clusterDim.z = 1;
    }
    if (behind) {
        cudaLaunchAttribute &c = at[cfg.numAttrs++];
        c.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        c.val.programmaticStreamSerializationAllowed = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, p...);
}

inline int32_t ceil_div(int64_t a, int64_t b) { return static_cast<int32_t>((a + b - 1) / b); }

}  // namespace harts
