// Launches that overlap their start with the end of the kernel before them on the
// stream (programmatic dependent launch): the CTAs are set up while that kernel's last
// ones still run, and wait in after_previous() until it is done and its results can be
// seen.  About 2 us a launch on GB300, where a kernel of the operators on rows takes 4
// to 100.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

namespace mk {

// the next kernel's CTAs may be set up (once all of this one's have begun)
__device__ __forceinline__ void allow_next() { cudaTriggerProgrammaticLaunchCompletion(); }

// first statement of a kernel that launch_early() launches: nothing that another kernel
// writes is read, and nothing that it reads is written, before
__device__ __forceinline__ void after_previous() {
    allow_next();
    cudaGridDependencySynchronize();
}

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, A&&... args) {
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = s;
    config.attrs = &early;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, kernel, static_cast<A&&>(args)...);
}

}  // namespace mk
