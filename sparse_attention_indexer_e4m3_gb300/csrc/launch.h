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
struct PageTable;
struct StepMapArgs;
struct PagedAttnParams;
struct VerifyArgs;

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

// bf16 paged cache: attention (D in {64, 128, 256, 512}) by `grid` CTAs and the join of the units that they share; its
// maps' boxes are [64 dims][p.box_rows] (a page's rows, paged_attn_block(D) at most) and [64 dims][paged_attn_cols(D)].
cudaError_t launch_paged_attn(int D, int grid, const CUtensorMap& kvmap, const CUtensorMap& qmap, const PagedAttnParams& p,
                              unsigned* err, cudaStream_t stream);
int paged_attn_smem(int D);
int paged_attn_cols(int D);   // most columns (token, head) of a unit
int paged_attn_block(int D);  // rows of a block
constexpr int kPagedMaxTokens = 32;  // most tokens of a unit
// A step's tokens from the sequences' lengths; packed keys to rows of the pages; bf16 rows into their pages.
cudaError_t launch_step_maps(const StepMapArgs& a, cudaStream_t stream);
cudaError_t launch_page_slots(const PageTable& c, const int32_t* seq, const int32_t* start, const int32_t* idx, int T, int K,
                              int32_t* slots, cudaStream_t stream);
cudaError_t launch_store_kv(int D, const uint16_t* kv, int64_t stride, int N, const int32_t* seq, const int32_t* pos,
                            const int32_t* lacking, uint16_t* pages, const PageTable& c, cudaStream_t stream);
// Drafted tokens against the target's probabilities, by clusters of CTAs.
cudaError_t launch_verify_drafts(const VerifyArgs& a, int sms, cudaStream_t stream);
// 2-D map over a row-major bf16 matrix [rows, D], box [64 dims][box_rows], 128-byte swizzle; false where it cannot be made.
bool make_bf16_map(CUtensorMap* map, const void* base, int64_t rows, int D, int box_rows);

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
