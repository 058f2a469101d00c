// pdl.cuh - programmatic dependent launch: a kernel of one call that starts
// while the one before it in the stream still runs, and waits inside for what
// that one leaves.  Only kernels after the first of a call are launched so: the
// first waits for all earlier work of the stream, as usual.
#pragma once

#include <cuda_runtime.h>

namespace vdn {

// Lets the next kernel of the call start (its CTAs as SMs have room).
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Waits until the kernels before have completed and their stores are visible.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<A&&>(args)...);
}

}  // namespace vdn
