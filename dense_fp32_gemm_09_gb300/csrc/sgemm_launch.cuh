// Launch as a programmatic dependent of the stream's previous kernel: the kernel may start
// while that one drains and waits (griddepcontrol.wait) before it touches global memory.
#pragma once

#include <cuda_runtime.h>

namespace sgemm {

__device__ __forceinline__ void wait_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void launch_next() {
    asm volatile("griddepcontrol.launch_dependents;");
}

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                             cudaStream_t stream, A&&... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(static_cast<unsigned>(threads));
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

}  // namespace sgemm
