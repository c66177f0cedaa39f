// Launches of the single-token kernels.
//
// A token's kernels are short (2 to 10 us), so the gap between one's end and the next one's start is a good part of
// their time. They are launched with programmatic stream serialization: a kernel's CTAs may be set up while the kernel
// before it still runs, and each thread then waits for that one's end (and its writes) before it touches memory.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace kda {

// What is asked of a device once and kept, by its number: a whole launch takes 1.6 us.
constexpr int kDevices = 32;
constexpr int kGb300Sms = 152;

// The present device, or -1 without one.
inline int present_device() {
    int device;
    return cudaGetDevice(&device) == cudaSuccess ? device : -1;
}

// SMs of the device; without one, those of a GB300.
inline int sm_count(int device) {
    static std::atomic<int> known[kDevices];
    int n = 0;
    if (device < 0) return kGb300Sms;
    if (device < kDevices && (n = known[device].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n <= 0) return kGb300Sms;
    if (device < kDevices) known[device].store(n, std::memory_order_relaxed);
    return n;
}
inline int sm_count() { return sm_count(present_device()); }

// The largest cluster, of at most `most` CTAs, that the device, which is the present one, can place the kernel in
// (without one: `most`). `known` is the kernel's own.
inline int largest_cluster(int device, const void* kernel, int threads, int most, std::atomic<int> (&known)[kDevices],
                           size_t shared = 0) {
    int n = 0;
    if (device < 0) return most;
    if (device < kDevices && (n = known[device].load(std::memory_order_relaxed)) > 0) return n;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(most);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxPotentialClusterSize(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = 1;
    }
    if (n > most) n = most;
    if (device < kDevices) known[device].store(n, std::memory_order_relaxed);
    return n;
}

// Division of numbers below 2^31 by an invariant d (Granlund and Montgomery, 1994): with 2^s >= d, floor(n / d) =
// floor(n ceil(2^(31 + s) / d) / 2^(31 + s)).
struct Divisor {
    unsigned factor, shift;
    Divisor() = default;
    __host__ explicit Divisor(unsigned d) : shift(31 + (d > 1 ? 32 - __builtin_clz(d - 1) : 0)) {
        factor = (unsigned)(((1ull << shift) + d - 1) / d);
    }
    __device__ __forceinline__ unsigned operator()(unsigned n) const {
        return (unsigned)((uint64_t)n * factor >> shift);
    }
};

// Every thread of a kernel launched by launch_after calls this first, whatever it does then: a kernel that ended
// without having waited would let the one after it start before the one before it has ended.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A cluster of more than 8 CTAs is one that largest_cluster allowed on this device.
template <typename Args>
cudaError_t launch_after(void (*kernel)(Args), const Args& a, dim3 grid, int threads, cudaStream_t st,
                         int cluster = 1, size_t shared = 0) {
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace kda
