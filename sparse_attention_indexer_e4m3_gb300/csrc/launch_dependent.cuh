// Launch of a kernel that waits for the stream's earlier work itself.
#pragma once

#include <cuda_runtime.h>

namespace dsa {

// The kernel begins with griddepcontrol.wait: its own way onto the SMs then overlaps the end of the kernel before it,
// which a decoding step's small calls are mostly made of.
template <class... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, unsigned block, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(block);
  c.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace dsa
