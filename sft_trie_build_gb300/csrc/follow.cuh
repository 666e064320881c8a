// Kernels of one call that follow one another: the second one's launch does not
// wait for the first one's end, only its reads do.
#pragma once

#include <cuda_runtime.h>

namespace stp {

// First in a kernel that launch_after starts: what the kernel before it in the
// stream has written can be read behind this.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches `kernel`, which begins with wait_for_previous, behind a kernel of the same call.
template <typename P>
cudaError_t launch_after(void (*kernel)(P), dim3 grid, dim3 block, cudaStream_t s, P params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  void* args[] = {&params};
  return cudaLaunchKernelExC(&cfg, (const void*)kernel, args);
}

}  // namespace stp
