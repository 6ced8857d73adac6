// Launches that start while the kernel before them in the stream ends.
#pragma once
#include <cuda_runtime.h>

namespace moe {

// First thing in a kernel of launch_early, by every thread: all that came before in the stream is done and seen.
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... Q>
cudaError_t launch_early(void (*kernel)(P...), int grid, int block, size_t smem, cudaStream_t s, const Q&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace moe
