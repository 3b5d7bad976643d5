// Launches of the serving kernels.  Each may be launched while the kernel before
// it in the stream still runs (programmatic dependent launch), so that a decode
// step's short kernels do not pay for a start each; none touches memory before
// wait_for_previous, unless its launcher says why it may.
#pragma once

#include <cuda_runtime.h>

namespace dhsa {

// Lets the next kernel of the stream be launched early.  Given by every CTA of a
// kernel, or by its exit.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Returns when the kernel before in the stream has completed and its writes are
// visible (at once where this kernel was not launched early).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream,
                         const A&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace dhsa
