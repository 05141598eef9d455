// Sparse attention over the 4-bit paged cache: launcher (its own translation unit, compiled in parallel
// with the others).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "attn_kv4_kernel.cuh"
#include "launch.h"

namespace dsa {

namespace {

constexpr int kDevices = 64;

// Shared memory and cluster size of the kernel on the current device, set once per device (setting them again, from
// another thread too, changes nothing), and how many clusters of `shares` CTAs the device runs at a time: 0 for a
// size that it does not run, negative on a CUDA error.
template <int D>
int clusters_d(int shares) {
  static std::atomic<int> known[kDevices][kKv4MaxShares + 1];  // by cluster size: clusters + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return -1;
  const int have = known[dev][shares].load(std::memory_order_acquire);
  if (have > 0) return have - 1;
  constexpr int smem = AttnKv4Layout<D>::kSmem;
  if (cudaFuncSetAttribute(sparse_attn_kv4_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(sparse_attn_kv4_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaFuncSetAttribute(sparse_attn_kv4_kernel<D, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return -1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(static_cast<unsigned>(shares));
  c.blockDim = dim3(kKv4Threads);
  c.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(shares);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  int clusters = shares == 1 ? 1 : 0;
  if (shares > 1 && cudaOccupancyMaxActiveClusters(&clusters, sparse_attn_kv4_kernel<D, true>, &c) != cudaSuccess) {
    (void)cudaGetLastError();
    clusters = 0;
  }
  known[dev][shares].store(clusters + 1, std::memory_order_release);
  return clusters;
}

template <int D>
cudaError_t launch_d(int grid, int shares, const AttnKv4Params& p, unsigned* err, cudaStream_t stream) {
  if (clusters_d<D>(shares) < 1) return cudaErrorInvalidValue;
  // every unit on a CTA or cluster of its own, or one CTA walking over several
  const bool single = static_cast<int64_t>(p.T) * p.groups * shares == grid;
  if (!single && shares > 1) return cudaErrorInvalidValue;
  const auto kernel = single ? sparse_attn_kv4_kernel<D, true> : sparse_attn_kv4_kernel<D, false>;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(static_cast<unsigned>(grid));
  c.blockDim = dim3(kKv4Threads);
  c.dynamicSmemBytes = AttnKv4Layout<D>::kSmem;
  c.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(shares);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (the kernel waits for the stream itself)
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, kernel, p, shares, err);
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

int sparse_attn_kv4_clusters(int D, int shares) {
  switch (D) {
    case 64: return clusters_d<64>(shares);
    case 128: return clusters_d<128>(shares);
    case 256: return clusters_d<256>(shares);
    case 512: return clusters_d<512>(shares);
    default: return -1;
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
