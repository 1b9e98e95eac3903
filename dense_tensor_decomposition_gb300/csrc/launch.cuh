// Launches that overlap their start with the end of the kernel before them on the
// stream (programmatic dependent launch): the launch is set up before that kernel is
// done, and its CTAs wait in after_previous() until its results can be seen.  About 2 us
// a launch on GB300, where a kernel of the operators on rows takes 4 to 100.  The kernels
// do not allow the next one's CTAs before they are done themselves: CTAs that wait on an
// SM cost the running ones more (a CP gradient of 41611 samples, order 5, R = 8: 117 us
// so, 58 without).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

namespace mk {

// first statement of a kernel that launch_early() launches: nothing that another kernel
// writes is read, and nothing that it reads is written, before
__device__ __forceinline__ void after_previous() { cudaGridDependencySynchronize(); }

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
    const cudaError_t e = cudaLaunchKernelEx(&config, kernel, static_cast<A&&>(args)...);
    if (e != cudaSuccess) cudaGetLastError();       // the error is told by this call alone
    return e;
}

}  // namespace mk
