// The C ABI of the 4-bit paged cache (declared in include/dsa.h): argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/dsa.h"
#include "api_checks.h"
#include "kv4.cuh"
#include "launch.h"

namespace dsa {
namespace {

// The checks that the calls on a pool share; fills `c`.
dsa_status check_pool(Kv4Pool* c, const uint8_t* cache, int P, int page_rows, const int32_t* table, int R, int M, int D) {
  if (P < 0 || R < 0 || M < 0) return DSA_ERR_INVALID_ARG;
  if (!paged_d(D) || !paged_rows(page_rows)) return DSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(M) * page_rows > INT_MAX) return DSA_ERR_UNSUPPORTED;  // a row's position is an int
  if (P > 0 && (!cache || !aligned(cache, 16))) return DSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(R) * M > 0 && (!table || !aligned(table, 4))) return DSA_ERR_INVALID_ARG;
  *c = Kv4Pool{const_cast<uint8_t*>(cache), table, P, R, M, log2_of(page_rows)};
  return DSA_OK;
}

dsa_status check_tables(int R, int M, int P) {
  if (R < 0 || M < 0 || P < 0) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

// Longest list.  A list's last entry is looked for from its end, 256 entries at a time, while the other roles of the
// kernel wait for it: with nothing but -1 behind its first entry that takes 0.2 s at this length (a wait expires after 1 s).
constexpr int kKv4MaxList = 1 << 26;

int head_groups(int H) { return H / kTcMaxHeads + (H % kTcMaxHeads != 0 ? 1 : 0); }

// CTAs that share a unit's list: as few blocks per share as the device has clusters for, all units at once.  Joining the shares
// takes as long as two to three blocks do, so a list is shared where at least that many of its blocks go to other CTAs
// (one token, 64 heads, in a graph, shared against not: 4 blocks, D = 64 9.4 to 10.8 us, 128 9.6 to 10.8, 256 11.6 to 13.2,
// 512 14.9 to 19.5; 16 blocks 10.6 to 23.8, 10.8 to 24.0, 12.1 to 32.2, 15.2 to 54.1; 3 blocks at D = 512 15.8 to 16.6).
int list_shares(int64_t units, int D, int K) {
  const int blocks = K / kKv4Block + (K % kKv4Block != 0 ? 1 : 0);
  const int worth = D == 512 ? 2 : 3;
  if (blocks <= worth || units > sparse_attn_kv4_clusters(D, 2)) return 1;
  for (int most = std::min(blocks, kKv4MaxShares); most > 1; --most) {
    const int each = (blocks + most - 1) / most;
    if (blocks - each < worth) break;
    const int shares = (blocks + each - 1) / each;  // no more than it takes for `each` blocks per share
    if (units <= sparse_attn_kv4_clusters(D, shares)) return shares;
  }
  return 1;
}

size_t partial_bytes(int64_t units, int shares, int D) {
  return shares > 1 ? static_cast<size_t>(units) * shares * kTcMaxHeads * (D + 2) * sizeof(float) : 0;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

size_t dsa_kv4_page_bytes(int page_rows, int D) {
  return paged_d(D) && paged_rows(page_rows) ? static_cast<size_t>(page_rows) * kv4_row_bytes(D) : 0;
}

dsa_status dsa_quantize_kv4(const uint16_t* kv, const int32_t* seq, const int32_t* pos, int N, int D, uint8_t* cache,
                            int P, int page_rows, const int32_t* table, int R, int M, void* stream) {
  return dsa_quantize_kv4_reserved(kv, seq, pos, N, D, cache, P, page_rows, table, R, M, nullptr, stream);
}

dsa_status dsa_quantize_kv4_reserved(const uint16_t* kv, const int32_t* seq, const int32_t* pos, int N, int D,
                                     uint8_t* cache, int P, int page_rows, const int32_t* table, int R, int M,
                                     const int32_t* lacking, void* stream) {
  Kv4Pool c;
  const dsa_status st = check_pool(&c, cache, P, page_rows, table, R, M, D);
  if (st != DSA_OK) return st;
  if (N < 0) return DSA_ERR_INVALID_ARG;
  if (N == 0) return DSA_OK;
  if (!kv || !aligned(kv, 32) || !seq || !aligned(seq, 4) || !pos || !aligned(pos, 4)) return DSA_ERR_INVALID_ARG;
  if (lacking && !aligned(lacking, 4)) return DSA_ERR_INVALID_ARG;
  return done(launch_kv4_write(D, kv, N, seq, pos, lacking, c, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_dequantize_kv4(const uint8_t* cache, int P, int page_rows, const int32_t* table, int R, int M,
                              const int32_t* seq, const int32_t* pos, int N, int D, uint16_t* kv, void* stream) {
  Kv4Pool c;
  const dsa_status st = check_pool(&c, cache, P, page_rows, table, R, M, D);
  if (st != DSA_OK) return st;
  if (N < 0) return DSA_ERR_INVALID_ARG;
  if (N == 0) return DSA_OK;
  if (!kv || !aligned(kv, 32) || !seq || !aligned(seq, 4) || !pos || !aligned(pos, 4)) return DSA_ERR_INVALID_ARG;
  return done(launch_kv4_read(D, kv, N, seq, pos, c, static_cast<cudaStream_t>(stream)));
}

size_t dsa_sparse_attn_kv4_workspace_size(int T, int H, int D, int K) {
  if (T <= 0 || H < 1 || K <= 0 || !paged_d(D)) return 0;
  const int64_t units = static_cast<int64_t>(T) * head_groups(H);
  return partial_bytes(units, list_shares(units, D, K), D);
}

dsa_status dsa_sparse_attn_kv4(const uint16_t* q, const uint8_t* cache, int P, int page_rows, const int32_t* table,
                               int R, int M, const int32_t* seq, const int32_t* start, const float* attn_sink,
                               const int32_t* idx, int T, int H, int D, int K, float scale, uint16_t* out, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream) {
  Kv4Pool c;
  const dsa_status st = check_pool(&c, cache, P, page_rows, table, R, M, D);
  if (st != DSA_OK) return st;
  if (T < 0 || H < 1 || K < 0) return DSA_ERR_INVALID_ARG;
  if (T == 0) return DSA_OK;
  if (!q || !aligned(q, 16) || !out || !aligned(out, 16) || !seq || !aligned(seq, 4)) return DSA_ERR_INVALID_ARG;
  if (K > 0 && (!idx || !aligned(idx, 4))) return DSA_ERR_INVALID_ARG;
  if ((start && !aligned(start, 4)) || (attn_sink && !aligned(attn_sink, 4)) || (lse && !aligned(lse, 4)))
    return DSA_ERR_INVALID_ARG;
  const int groups = head_groups(H);
  const int64_t units = static_cast<int64_t>(T) * groups;
  if (units > INT_MAX / 2 || K > kKv4MaxList) return DSA_ERR_UNSUPPORTED;
  DeviceFacts dev;
  if (!device_facts(&dev)) return DSA_ERR_CUDA;
  if (sparse_attn_kv4_smem(D) > dev.max_smem) return DSA_ERR_UNSUPPORTED;
  const int shares = list_shares(units, D, K);
  if (shares > 1 && (!workspace || !aligned(workspace, 16) || workspace_bytes < partial_bytes(units, shares, D)))
    return DSA_ERR_WORKSPACE;
  const int grid = shares > 1 ? static_cast<int>(units) * shares : static_cast<int>(std::min<int64_t>(units, dev.sms));
  float* partial = shares > 1 ? static_cast<float*>(workspace) : nullptr;
  float* stats = shares > 1 ? partial + units * shares * kTcMaxHeads * D : nullptr;
  const AttnKv4Params p{q, c, seq, start, attn_sink, idx, out, lse, partial, stats, T, H, K, groups, scale};
  return done(launch_sparse_attn_kv4(D, grid, shares, p, dev.err, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_fork_pages(const int32_t* table, const int32_t* parent, int R, int M, int P, int32_t* ref,
                          int32_t* table_out, void* stream) {
  const dsa_status st = check_tables(R, M, P);
  if (st != DSA_OK) return st;
  const int64_t entries = static_cast<int64_t>(R) * M;
  if (entries == 0) return DSA_OK;
  if (!table || !aligned(table, 4) || !parent || !aligned(parent, 4) || !table_out || !aligned(table_out, 4) ||
      (P > 0 && (!ref || !aligned(ref, 4))))
    return DSA_ERR_INVALID_ARG;
  // rows are read while others are written: the two tables must not overlap
  const uintptr_t a = reinterpret_cast<uintptr_t>(table), b = reinterpret_cast<uintptr_t>(table_out);
  const uintptr_t bytes = static_cast<uintptr_t>(entries) * 4;
  if (a < b + bytes && b < a + bytes) return DSA_ERR_INVALID_ARG;
  return done(launch_pages_fork(table, parent, R, M, P, ref, table_out, static_cast<cudaStream_t>(stream)));
}

size_t dsa_reserve_pages_workspace_size(int P) { return P > 0 ? static_cast<size_t>(P) * 8 : 0; }

dsa_status dsa_reserve_pages(int32_t* table, int32_t* ref, const int32_t* begin, const int32_t* end, int R, int M, int P,
                             int page_rows, int32_t* src, int32_t* dst, int32_t* lacking, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const dsa_status st = check_tables(R, M, P);
  if (st != DSA_OK) return st;
  if (!paged_rows(page_rows) || static_cast<int64_t>(M) * page_rows > INT_MAX || R > INT_MAX / 2) return DSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(R) * M > INT_MAX) return DSA_ERR_UNSUPPORTED;  // as many needs at most, which are counted in ints
  if (!lacking || !aligned(lacking, 4)) return DSA_ERR_INVALID_ARG;
  if (R > 0 && (!begin || !aligned(begin, 4) || !end || !aligned(end, 4) || !src || !aligned(src, 4) || !dst ||
                !aligned(dst, 4)))
    return DSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(R) * M > 0 && (!table || !aligned(table, 4))) return DSA_ERR_INVALID_ARG;
  if (P > 0 && (!ref || !aligned(ref, 4))) return DSA_ERR_INVALID_ARG;
  if (P > 0 && (!workspace || !aligned(workspace, 4) || workspace_bytes < dsa_reserve_pages_workspace_size(P)))
    return DSA_ERR_WORKSPACE;
  int32_t* ws = static_cast<int32_t*>(workspace);
  const ReserveArgs a{table, ref, begin, end, R, M, P, log2_of(page_rows), src, dst, lacking, ws, ws + P};
  return done(launch_pages_reserve(a, static_cast<cudaStream_t>(stream)));
}

size_t dsa_compact_pages_workspace_size(int P) { return P > 0 ? static_cast<size_t>(P) * 4 : 0; }

dsa_status dsa_compact_pages(int32_t* table, int32_t* ref, int R, int M, int P, int32_t* src, int32_t* dst,
                             int32_t* n_live, void* workspace, size_t workspace_bytes, void* stream) {
  const dsa_status st = check_tables(R, M, P);
  if (st != DSA_OK) return st;
  const int64_t entries = static_cast<int64_t>(R) * M;
  if (!n_live || !aligned(n_live, 4)) return DSA_ERR_INVALID_ARG;
  if (entries > 0 && (!table || !aligned(table, 4))) return DSA_ERR_INVALID_ARG;
  if (P > 0 && (!ref || !aligned(ref, 4))) return DSA_ERR_INVALID_ARG;
  if (P > 1 && (!src || !aligned(src, 4) || !dst || !aligned(dst, 4))) return DSA_ERR_INVALID_ARG;
  if (P > 0 && (!workspace || !aligned(workspace, 4) || workspace_bytes < dsa_compact_pages_workspace_size(P)))
    return DSA_ERR_WORKSPACE;
  const CompactArgs a{ref, P, src, dst, n_live, static_cast<int32_t*>(workspace), nullptr, 0};
  return done(launch_pages_compact(a, table, entries, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_copy_pages(void* pages, size_t page_bytes, int P, const int32_t* src, const int32_t* dst, int n,
                          void* stream) {
  if (P < 0 || n < 0) return DSA_ERR_INVALID_ARG;
  if (page_bytes == 0 || page_bytes % 16 != 0 || page_bytes > (static_cast<size_t>(1) << 40)) return DSA_ERR_UNSUPPORTED;
  if (n == 0 || P == 0) return DSA_OK;
  if (!pages || !aligned(pages, 16) || !src || !aligned(src, 4) || !dst || !aligned(dst, 4)) return DSA_ERR_INVALID_ARG;
  DeviceFacts dev;
  if (!device_facts(&dev)) return DSA_ERR_CUDA;
  return done(launch_pages_copy(static_cast<uint8_t*>(pages), static_cast<int64_t>(page_bytes), P, src, dst, n, dev.sms,
                                static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
