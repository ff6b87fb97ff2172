// launch.cuh -- launches that may begin while the kernel before them on the
// stream ends. Each step kernel calls grid_begin() before it touches memory: it
// lets the next such launch be set up, and waits until everything before it on
// the stream is complete and visible. Inputs are read by plain loads: one marked
// as reading what never changes (__ldg, const __restrict__) could be moved in
// front of the wait. What is saved is the set-up between two
// kernels, 1 to 2 us, as much as the smallest of them take.
#pragma once

#include <cuda_runtime.h>

namespace tpce {
namespace step {

__device__ __forceinline__ void grid_begin() {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace step
}  // namespace tpce
