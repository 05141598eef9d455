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
  const int pieces = K / kSlotEach + (K % kSlotEach != 0 ? 1 : 0);
  const bool wide = K % kSlotEach == 0 && (reinterpret_cast<uintptr_t>(idx) & 15) == 0 && (reinterpret_cast<uintptr_t>(slots) & 15) == 0;
  const int64_t blocks = (static_cast<int64_t>(T) * pieces + kSlotThreads - 1) / kSlotThreads;
  return launch_dependent(page_slots_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(blocks, 1 << 30))), kSlotThreads, stream, c, seq,
                          start, idx, T, K, slots, pieces, wide);
}

cudaError_t launch_store_kv(int D, const uint16_t* kv, int64_t stride, int N, const int32_t* seq, const int32_t* pos,
                            const int32_t* lacking, uint16_t* pages, const PageTable& c, cudaStream_t stream) {
  const int log_pieces = D == 64 ? 3 : D == 128 ? 4 : D == 256 ? 5 : 6;  // 16-byte pieces of a row
  const int64_t blocks = ((static_cast<int64_t>(N) << log_pieces) + kStoreThreads - 1) / kStoreThreads;
  return launch_dependent(store_kv_kernel, dim3(static_cast<unsigned>(blocks)), kStoreThreads, stream, kv, stride, N, log_pieces, seq, pos,
                          lacking, pages, c);
}

cudaError_t launch_verify_drafts(const VerifyArgs& a, int sms, cudaStream_t stream) {
  // CTAs of a row: as many as bring about two to every SM, each with a few pieces a warp at least
  int cluster = kVerMaxCluster;
  while (cluster > 1 && (static_cast<int64_t>(a.R) * cluster > 4 * sms || a.V / cluster < kVerPiece * kVerWarps)) cluster /= 2;
  int64_t piece = kVerPiece;
  while ((a.V + piece - 1) / piece > static_cast<int64_t>(kVerPieces) * cluster) piece *= 2;
  const int pieces = static_cast<int>((a.V + piece - 1) / piece);
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(static_cast<unsigned>(a.R) * cluster);
  c.blockDim = dim3(kVerThreads);
  c.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, verify_drafts_kernel, a, cluster, static_cast<int>(piece), pieces);
}

}  // namespace dsa
