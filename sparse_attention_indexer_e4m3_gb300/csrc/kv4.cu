// The 4-bit paged cache's codec and page calls: launchers (their own translation unit).
#include <cuda_runtime.h>

#include <algorithm>

#include "kv4_codec_kernel.cuh"
#include "launch.h"
#include "pages_kernel.cuh"

namespace dsa {

namespace {

template <int D>
unsigned codec_grid(int N) {
  return static_cast<unsigned>((static_cast<int64_t>(N) * (D / kKv4Group) + kKv4CodecThreads - 1) / kKv4CodecThreads);
}

// Launch of a kernel that waits for the stream's earlier work itself (griddepcontrol.wait): its own way onto the SMs
// then overlaps the end of the kernel before it, which a decoding step's small calls are mostly made of.
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

}  // namespace

#define DSA_KV4_BY_D(D, CALL)             \
  switch (D) {                            \
    case 64: CALL(64);                     \
    case 128: CALL(128);                   \
    case 256: CALL(256);                   \
    case 512: CALL(512);                   \
    default: return cudaErrorInvalidValue; \
  }

cudaError_t launch_kv4_write(int D, const uint16_t* x, int N, const int32_t* seq, const int32_t* pos, const int32_t* lacking,
                             const Kv4Pool& c, cudaStream_t stream) {
#define DSA_CALL(DD) return launch_dependent(kv4_write_kernel<DD>, dim3(codec_grid<DD>(N)), kKv4CodecThreads, stream, x, N, seq, pos, lacking, c)
  DSA_KV4_BY_D(D, DSA_CALL)
#undef DSA_CALL
}

cudaError_t launch_kv4_read(int D, uint16_t* out, int N, const int32_t* seq, const int32_t* pos, const Kv4Pool& c,
                            cudaStream_t stream) {
#define DSA_CALL(DD) return launch_dependent(kv4_read_kernel<DD>, dim3(codec_grid<DD>(N)), kKv4CodecThreads, stream, out, N, seq, pos, c)
  DSA_KV4_BY_D(D, DSA_CALL)
#undef DSA_CALL
}

cudaError_t launch_pages_fork(const int32_t* table, const int32_t* parent, int R, int M, int P, int32_t* ref,
                              int32_t* out, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(std::min((static_cast<int64_t>(M) + 255) / 256, static_cast<int64_t>(1) << 16)),
                  static_cast<unsigned>(std::min(R, 65535)));
  return launch_dependent(pages_fork_kernel, grid, 256u, stream, table, parent, R, M, P, ref, out);
}

cudaError_t launch_pages_reserve(const ReserveArgs& a, cudaStream_t stream) {
  return launch_dependent(pages_reserve_kernel, dim3(kPagesCluster), kPagesThreads, stream, a);
}

cudaError_t launch_pages_compact(CompactArgs a, int32_t* table, int64_t entries, cudaStream_t stream) {
  // A small table in the same launch, a large one over all SMs in a second (16384 pages: 450 entries 7.6 to 7.9 us, 16384
  // entries 8.0 to 8.0, 65536 9.3 to 8.5, 1 M 24.7 to 11.6; the second launch also costs the host 2 us).
  constexpr int64_t kSmallTable = 1 << 14;
  const bool small = entries <= kSmallTable;
  a.table = small ? table : nullptr;
  a.entries = small ? static_cast<int>(entries) : 0;
  const cudaError_t e = launch_dependent(pages_compact_kernel, dim3(kPagesCluster), kPagesThreads, stream, static_cast<const CompactArgs>(a));
  if (e != cudaSuccess || small) return e;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((entries + 255) / 256, 1 << 16));
  return launch_dependent(pages_relabel_kernel, dim3(grid), 256u, stream, table, entries, a.P, static_cast<const int32_t*>(a.remap));
}

cudaError_t launch_pages_copy(uint8_t* pages, int64_t page_bytes, int P, const int32_t* src, const int32_t* dst, int n,
                              int sms, cudaStream_t stream) {
  const int64_t pieces = (page_bytes + kCopyPiece - 1) / kCopyPiece;
  const int grid = static_cast<int>(std::min<int64_t>(n * pieces, static_cast<int64_t>(sms) * 8));
  return launch_dependent(pages_copy_kernel, dim3(grid), kCopyThreads, stream, pages, page_bytes, P, src, dst, n,
                          static_cast<int>(pieces));
}

}  // namespace dsa
