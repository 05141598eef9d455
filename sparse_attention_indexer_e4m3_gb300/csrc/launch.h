// Host-side launchers of the library's kernels (one translation unit per head dimension and
// one for the selection kernels, so they compile in parallel).  Internal to the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dsa {

struct IndexParams;
struct TopkParams;
struct PlanArgs;
struct AttnParams;
struct AttnBwdParams;
struct KresParams;
struct AttnKv4Params;
struct Kv4Pool;
struct ReserveArgs;
struct CompactArgs;

// Index kernel for head dimension 128 / 64; `fused` selects the fused index + top-k mode.
cudaError_t launch_index_d128(int H, bool fused, int grid, size_t smem, cudaStream_t stream, const CUtensorMap& kmap,
                              const CUtensorMap& qmap, const IndexParams& p);
cudaError_t launch_index_d64(int H, bool fused, int grid, size_t smem, cudaStream_t stream, const CUtensorMap& kmap,
                             const CUtensorMap& qmap, const IndexParams& p);

// K-resident scorer (window pass, then the scorer) for head dimension 128 / 64.
cudaError_t launch_kres_d128(int H, int grid, size_t smem, cudaStream_t stream, const CUtensorMap& kmap,
                             const CUtensorMap& qmap, const KresParams& p, const int32_t* ks, const int32_t* ke);
cudaError_t launch_kres_d64(int H, int grid, size_t smem, cudaStream_t stream, const CUtensorMap& kmap,
                            const CUtensorMap& qmap, const KresParams& p, const int32_t* ks, const int32_t* ke);

cudaError_t launch_topk_rows(int grid, size_t smem, cudaStream_t stream, const TopkParams& p);
// Streaming top-k for rows of at most kTopkStreamMaxKeys keys; as many CTAs as fit, <= max_grid.
cudaError_t launch_topk_stream(int max_grid, size_t smem, cudaStream_t stream, const TopkParams& p);
cudaError_t launch_plan(cudaStream_t stream, const PlanArgs& a);
// e4m3 quantise-on-write of N rows of D (64 or 128) bf16 values.
cudaError_t launch_quantize(int D, const uint16_t* x, int64_t N, uint8_t* codes, float* scale, cudaStream_t stream);
// One CTA exercising the bounded wait on barriers that never complete (about kWaitLimitNs).
cudaError_t launch_wait_check(cudaStream_t stream, unsigned* err, unsigned long long* took_ns);

// Sparse attention over the selected keys, head dimension D (64, 128, 256 or 512): CUDA cores.
cudaError_t launch_sparse_attn(int D, const AttnParams& p, cudaStream_t stream);
// Heads one tensor-core attention launch takes (the N of its products); a layer with more heads
// runs as groups of at most this many, each a launch over the same lists (p.hs = the layer's heads).
constexpr int kTcMaxHeads = 64;
// The same on the tensor cores (D in {128, 256, 512}, H <= kTcMaxHeads, q and kv 16-byte
// aligned): `grid` persistent CTAs over the query rows; its bounded waits record into *err.
// Dynamic shared memory it needs (0 for an unsupported D).
cudaError_t launch_sparse_attn_tc(int D, int grid, const AttnParams& p, unsigned* err, cudaStream_t stream);
int sparse_attn_tc_smem(int D);
// Gradients of the sparse attention on the tensor cores (D in {128, 256}, H <= kTcMaxHeads): `grid`
// persistent CTAs over the query rows; dkv and dsink must be zeroed first.
cudaError_t launch_sparse_attn_bwd_tc(int D, int grid, const AttnBwdParams& p, unsigned* err, cudaStream_t stream);
int sparse_attn_bwd_tc_smem(int D);

// 4-bit paged cache: N rows of D (64, 128, 256 or 512) bf16 values into their pages and back.
// (into: nothing is written where *lacking is given and not 0).
cudaError_t launch_kv4_write(int D, const uint16_t* x, int N, const int32_t* seq, const int32_t* pos, const int32_t* lacking,
                             const Kv4Pool& c, cudaStream_t stream);
cudaError_t launch_kv4_read(int D, uint16_t* out, int N, const int32_t* seq, const int32_t* pos, const Kv4Pool& c,
                            cudaStream_t stream);
// Page tables: rows from their parents, pages for rows about to be written, live pages to the front, copies.
cudaError_t launch_pages_fork(const int32_t* table, const int32_t* parent, int R, int M, int P, int32_t* ref,
                              int32_t* out, cudaStream_t stream);
cudaError_t launch_pages_reserve(const ReserveArgs& a, cudaStream_t stream);
cudaError_t launch_pages_compact(CompactArgs a, int32_t* table, int64_t entries, cudaStream_t stream);
cudaError_t launch_pages_copy(uint8_t* pages, int64_t page_bytes, int P, const int32_t* src, const int32_t* dst, int n,
                              int sms, cudaStream_t stream);
// Sparse attention over the 4-bit paged cache (D in {64, 128, 256, 512}); `shares` CTAs of a cluster
// share a unit's list.
constexpr int kKv4Block = 128;     // list entries per block
constexpr int kKv4MaxShares = 16;  // most CTAs that share a list
cudaError_t launch_sparse_attn_kv4(int D, int grid, int shares, const AttnKv4Params& p, unsigned* err,
                                   cudaStream_t stream);
int sparse_attn_kv4_smem(int D);
// How many clusters of `shares` of its CTAs this device runs at a time (0: none of that size; < 0: a CUDA error).
int sparse_attn_kv4_clusters(int D, int shares);

// Facts of the current device that the entry points need; false on a CUDA error.
struct DeviceFacts {
  int sms;
  int max_smem;
  unsigned* err;  // the device error word
};
bool device_facts(DeviceFacts* f);

// Largest dynamic shared memory a CTA of this device may use (bytes).
int max_dynamic_smem();

}  // namespace dsa
