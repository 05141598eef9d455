// Attention over the bf16 paged cache: launcher (its own translation unit).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "launch.h"
#include "paged_attn_kernel.cuh"

namespace dsa {

namespace {

constexpr int kDevices = 64;

template <int D>
cudaError_t launch_d(int grid, const CUtensorMap& kvmap, const CUtensorMap& qmap, const PagedAttnParams& p, unsigned* err,
                     cudaStream_t stream) {
  static std::atomic<bool> set[kDevices];  // (setting it again, from another thread too, changes nothing)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  if (!set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(paged_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PagedLayout<D>::kSmem);
    if (e != cudaSuccess) return e;
    set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(static_cast<unsigned>(grid));
  c.blockDim = dim3(PagedLayout<D>::kThreads);
  c.dynamicSmemBytes = PagedLayout<D>::kSmem;
  c.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (the kernels wait for the stream themselves)
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, paged_attn_kernel<D>, kvmap, qmap, p, err);
  if (e != cudaSuccess || grid == 1) return e;  // (one CTA shares nothing)
  // the shared units: an entry each, over eight blocks for each SM where they are few (as many as the cut that is expected has)
  const int entries = paged_entries(p, grid), items = std::max(p.whole.rows, p.any.rows) * std::max(1, D / 128);
  const int units = std::min(p.guess != 0 ? p.any.units : p.whole.units, grid);
  c.gridDim = dim3(static_cast<unsigned>(entries), static_cast<unsigned>(std::min(items, std::max(1, 8 * grid / units))));
  c.blockDim = dim3(kPgJoinThreads);
  c.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&c, paged_join_kernel<D>, p);
}

}  // namespace

int paged_attn_cols(int D) { return paged_cols(D); }
int paged_attn_block(int D) { return paged_block(D); }

int paged_attn_smem(int D) {
  switch (D) {
    case 64: return PagedLayout<64>::kSmem;
    case 128: return PagedLayout<128>::kSmem;
    case 256: return PagedLayout<256>::kSmem;
    case 512: return PagedLayout<512>::kSmem;
    default: return 0;
  }
}

cudaError_t launch_paged_attn(int D, int grid, const CUtensorMap& kvmap, const CUtensorMap& qmap, const PagedAttnParams& p,
                              unsigned* err, cudaStream_t stream) {
  switch (D) {
    case 64: return launch_d<64>(grid, kvmap, qmap, p, err, stream);
    case 128: return launch_d<128>(grid, kvmap, qmap, p, err, stream);
    case 256: return launch_d<256>(grid, kvmap, qmap, p, err, stream);
    case 512: return launch_d<512>(grid, kvmap, qmap, p, err, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dsa
