// Sparse attention over the 4-bit paged cache: launcher (its own translation unit, compiled in parallel
// with the others).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "attn_kv4_kernel.cuh"
#include "launch.h"

namespace dsa {

namespace {

template <int D>
cudaError_t launch_d(int grid, int shares, const AttnKv4Params& p, unsigned* err, cudaStream_t stream) {
  constexpr int smem = AttnKv4Layout<D>::kSmem;
  // once per device (setting it again, from another thread too, changes nothing)
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(sparse_attn_kv4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) set.fetch_or(uint64_t{1} << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(static_cast<unsigned>(grid));
  c.blockDim = dim3(kKv4Threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(shares);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, sparse_attn_kv4_kernel<D>, p, shares, err);
}

}  // namespace

int sparse_attn_kv4_smem(int D) {
  switch (D) {
    case 64: return AttnKv4Layout<64>::kSmem;
    case 128: return AttnKv4Layout<128>::kSmem;
    case 256: return AttnKv4Layout<256>::kSmem;
    case 512: return AttnKv4Layout<512>::kSmem;
    default: return 0;
  }
}

cudaError_t launch_sparse_attn_kv4(int D, int grid, int shares, const AttnKv4Params& p, unsigned* err,
                                   cudaStream_t stream) {
  switch (D) {
    case 64: return launch_d<64>(grid, shares, p, err, stream);
    case 128: return launch_d<128>(grid, shares, p, err, stream);
    case 256: return launch_d<256>(grid, shares, p, err, stream);
    case 512: return launch_d<512>(grid, shares, p, err, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dsa
