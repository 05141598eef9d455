// A serving step's small calls over the paged bf16 cache: launchers (their own translation unit).
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "launch_dependent.cuh"
#include "step_kernel.cuh"
#include "verify_kernel.cuh"

namespace dsa {

cudaError_t launch_step_maps(const StepMapArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.T) + kMapTokens - 1) / kMapTokens);
  return launch_dependent(step_maps_kernel, dim3(grid), kMapThreads, stream, a);
}

cudaError_t launch_page_slots(const PageTable& c, const int32_t* seq, const int32_t* start, const int32_t* idx, int T, int K,
                              int32_t* slots, cudaStream_t stream) {
  const bool wide = K % kSlotEach == 0 && (reinterpret_cast<uintptr_t>(idx) & 15) == 0 && (reinterpret_cast<uintptr_t>(slots) & 15) == 0;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(K) + kSlotThreads * kSlotEach - 1) / (kSlotThreads * kSlotEach)),
                  static_cast<unsigned>(std::min(T, 65535)));
  return launch_dependent(page_slots_kernel, grid, kSlotThreads, stream, c, seq, start, idx, T, K, slots, wide);
}

cudaError_t launch_store_kv(int D, const uint16_t* kv, int64_t stride, int N, const int32_t* seq, const int32_t* pos,
                            const int32_t* lacking, uint16_t* pages, const PageTable& c, cudaStream_t stream) {
  const int log_16 = D == 64 ? 3 : D == 128 ? 4 : D == 256 ? 5 : 6;  // 16-byte pieces of a row
  const bool wide = ((reinterpret_cast<uintptr_t>(kv) | reinterpret_cast<uintptr_t>(pages) | static_cast<uintptr_t>(2 * stride)) & 31) == 0;
  const int log_pieces = wide ? log_16 - 1 : log_16;
  const int64_t blocks = ((static_cast<int64_t>(N) << log_pieces) + kStoreThreads - 1) / kStoreThreads;
  return launch_dependent(wide ? store_kv_kernel<32> : store_kv_kernel<16>, dim3(static_cast<unsigned>(blocks)), kStoreThreads, stream, kv,
                          stride, N, log_pieces, seq, pos, lacking, pages, c);
}

cudaError_t launch_verify_drafts(const VerifyArgs& a, int sms, cudaStream_t stream) {
  // CTAs of a row: as many as are at work at a time, each with a few pieces a warp at least; larger ones where SMs are left over
  int cluster = kVerMaxCluster;
  while (cluster > 1 && (static_cast<int64_t>(a.R) * cluster > 2 * sms || a.V / cluster < kVerPiece * (kVerThreads / 32))) cluster /= 2;
  const bool large = static_cast<int64_t>(a.R) * cluster <= sms && a.V / cluster >= kVerPiece * (kVerMostThreads / 32);
  int64_t piece = kVerPiece;
  while ((a.V + piece - 1) / piece > static_cast<int64_t>(kVerPieces) * cluster) piece *= 2;
  const int pieces = static_cast<int>((a.V + piece - 1) / piece);
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(static_cast<unsigned>(a.R) * cluster);
  c.blockDim = dim3(large ? kVerMostThreads : kVerThreads);
  c.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, large ? verify_drafts_kernel<kVerMostThreads> : verify_drafts_kernel<kVerThreads>, a, cluster,
                            static_cast<int>(piece), pieces);
}

}  // namespace dsa
