// Launches of the single-token kernels.
//
// A token's kernels are short (2 to 10 us), so the gap between one's end and the next one's start is a good part of
// their time. They are launched with programmatic stream serialization: a kernel's CTAs may be set up while the kernel
// before it still runs, and each thread then waits for that one's end (and its writes) before it touches memory.
#pragma once
#include <cuda_runtime.h>

namespace kda {

// Every thread of a kernel launched by launch_after calls this first, whatever it does then: a kernel that ended
// without having waited would let the one after it start before the one before it has ended.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename Args>
cudaError_t launch_after(void (*kernel)(Args), const Args& a, dim3 grid, int threads, cudaStream_t st,
                         int cluster = 1) {
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    if (cluster > 8) {  // (the attribute stays with the kernel on its device: set it again only where that may differ)
        thread_local const void* set_for = nullptr;
        thread_local int set_on = -1;
        int device;
        cudaError_t e = cudaGetDevice(&device);
        if (e != cudaSuccess) return e;
        if (set_for != (const void*)kernel || set_on != device) {
            e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            set_for = (const void*)kernel;
            set_on = device;
        }
    }
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace kda
