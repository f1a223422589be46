// launch_after.cuh -- kernels of a step that start up while the kernel before them in the
// stream still runs (programmatic dependent launch).
//
// Such a kernel touches global memory only behind after_previous(), which returns when the
// kernel before it has completed and its writes are visible; that one waited in the same way
// for the one before it. (Loads are not those of the read-only path, __ldg: what they read
// must not change while the kernel runs, and it has started early.) What overlaps is the launch and the start of the blocks, and a
// following kernel of this kind may start up as soon as all blocks have got here. Copies,
// memsets and kernels launched in the ordinary way are ordered as ever. One call after the
// other: 8192 8-bit rows of 8 heads in and out 20.6 -> 16.3 us, an 8-bit decode step 26.8 ->
// 24.5, a drafting step over 16384 keys 101 -> 92.
#pragma once

#include <cuda_runtime.h>

namespace fanout {

__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    wait_for_previous();
}

// Launches `kernel`, which calls one of the two before it reads or writes anything.
template <typename... P>
cudaError_t launch_after(void (*kernel)(P...), int grid, int threads, int smem, cudaStream_t stream,
                         const P&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

}  // namespace fanout
