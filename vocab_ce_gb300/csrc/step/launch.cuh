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

// The same without letting the next launch begin: for a short kernel of few blocks,
// whose successor's blocks would find their places while the kernel before it
// still runs, on some SMs many and on others none.
__device__ __forceinline__ void grid_begin_alone() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A failed call's error, taken off the runtime's record as well: there the check after
// the next launch would find it, and report a kernel as failed that has run.
inline cudaError_t taken(cudaError_t e) {
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

// `ctas` neighbouring blocks form a cluster
template <typename... P, typename... A>
cudaError_t launch_clusters(int ctas, void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s,
                            const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    cudaGetLastError();  // what an earlier call has left there, and returned to its caller
    return taken(cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...));
}
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
    return launch_clusters(1, kernel, grid, threads, smem, s, args...);
}

}  // namespace step
}  // namespace tpce
