// Page tables of a paged cache: branching, growing, freeing and compacting sequences, and copying
// the pages that moved.
//
// The state is a table [R][M] of page ids (row = sequence; an id outside [0, P) is no page) and the
// counts ref[P] of the table entries that name each page; a page whose count is not positive is
// free, so no list of free pages is kept and every choice is the lowest free page.  All results are
// whole numbers and independent of scheduling (counts are summed with atomic adds, everything that
// is ranked is ranked by position).
//
// The calls that rank pages (reserve, compact) run as one cluster of eight CTAs: the counts are a few
// hundred KB at most, so a walk of them takes microseconds, and the cluster's hardware barrier and its
// distributed shared memory carry the prefix sums between the phases without further launches.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "cluster.cuh"
#include "kv4.cuh"

namespace dsa {

constexpr int kPagesCluster = 8;
constexpr int kPagesThreads = 1024;
constexpr int kPagesWarps = kPagesCluster * kPagesThreads / 32;  // warps of the cluster

// Contiguous share of warp g (of kPagesWarps) of n items, a multiple of 32 except for the last.
__device__ __forceinline__ void warp_share(int64_t n, int g, int64_t& lo, int64_t& hi) {
  const int64_t w = (n + kPagesWarps * 32 - 1) / (kPagesWarps * 32) * 32;
  lo = min(n, g * w);
  hi = min(n, lo + w);
}

// Per-warp counts of the cluster, two kinds: every warp publishes its own, the cluster's barrier, then
// every CTA's first kPagesWarps threads scan all of them.  `mine` receives the exclusive prefix of this warp,
// `total` the sums.
struct WarpCounts {
  int own[2][kPagesThreads / 32];
  int before[2][kPagesWarps];
  int part[2][kPagesWarps / 32];
  int total[2];
};

__device__ __forceinline__ void scan_warp_counts(WarpCounts& s, uint32_t rank, int c0, int c1, int (&mine)[2],
                                                 int (&total)[2]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    s.own[0][warp] = c0;
    s.own[1][warp] = c1;
  }
  cluster_sync_all();
  int v[2], x[2];
  if (threadIdx.x < kPagesWarps) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      v[k] = ld_cluster_s32(smem_addr(&s.own[k][lane]), static_cast<uint32_t>(warp));  // warp = rank read
      x[k] = v[k];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x[k], o);
        if (lane >= o) x[k] += y;
      }
      if (lane == 31) s.part[k][warp] = x[k];
    }
  }
  __syncthreads();
  if (threadIdx.x < kPagesWarps) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int base = 0;
      for (int w = 0; w < warp; ++w) base += s.part[k][w];
      s.before[k][threadIdx.x] = base + x[k] - v[k];
      if (threadIdx.x == kPagesWarps - 1) s.total[k] = base + x[k];
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    mine[k] = s.before[k][rank * (kPagesThreads / 32) + warp];
    total[k] = s.total[k];
  }
}

static_assert(kPagesThreads / 32 == 32 && kPagesWarps <= kPagesThreads, "one warp reads one CTA's counts");

// ---------------------------------------------------------------------------------------- fork

// out[r] = table[parent[r]] (no pages where parent[r] is outside [0, R)); ref follows the entries that
// change.  One thread per entry: the bytes of the two tables and of the counts bound it.
__global__ void __launch_bounds__(256) pages_fork_kernel(const int32_t* table,
                                                         const int32_t* parent, int R, int M, int P,
                                                         int32_t* ref, int32_t* out) {
  wait_stream();
  for (int r = blockIdx.y; r < R; r += gridDim.y) {
    const int p = ld_after_wait(parent + r);
    const int32_t* now = table + static_cast<int64_t>(r) * M;
    const bool some = static_cast<unsigned>(p) < static_cast<unsigned>(R);
    const int32_t* from = table + static_cast<int64_t>(some ? p : 0) * M;
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; j < M; j += static_cast<int64_t>(gridDim.x) * 256) {
      const int a = ld_after_wait(now + j);
      const int b = some ? ld_after_wait(from + j) : -1;
      out[static_cast<int64_t>(r) * M + j] = b;
      if (a != b) {
        if (static_cast<unsigned>(b) < static_cast<unsigned>(P)) atomicAdd(ref + b, 1);
        if (static_cast<unsigned>(a) < static_cast<unsigned>(P)) atomicSub(ref + a, 1);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------- reserve

// Page span [first, last] that rows [begin, end) of sequence r cover (last < first: none).
__device__ __forceinline__ void reserve_span(const ReserveArgs& a, int r, int64_t& b, int64_t& e, int& first, int& last) {
  b = max(0, ld_after_wait(a.begin + r));
  e = min(static_cast<int64_t>(ld_after_wait(a.end + r)), static_cast<int64_t>(a.M) << a.log_rows);
  first = 0;
  last = -1;
  if (e > b) {
    first = static_cast<int>(b >> a.log_rows);
    last = static_cast<int>((e - 1) >> a.log_rows);
  }
}

// Does entry `p` of a span need a page of its own: 0 no, 1 it has none, 2 its page is shared.
__device__ __forceinline__ int reserve_need(const ReserveArgs& a, int p) {
  if (static_cast<unsigned>(p) >= static_cast<unsigned>(a.P)) return 1;
  return a.ref[p] > 1 ? 2 : 0;
}

// Every page that rows [begin[r], end[r]) cover becomes mapped and sequence r's own.  All decisions go
// by the table and counts as they were at the call: (1) count the needs of each row and the free
// pages of each share of the counts; (2) the k-th lowest free page, for each k below the number of
// needs, into the workspace; (3) the k-th need, in the order of (r, page of r), takes the k-th page; (4) counts.
// A warp takes its rows one after another, so past a few hundred sequences the time grows with them (one row of each
// written, 64 pages a sequence: 64 sequences 8.5 us, 256 9.8, 1024 13.9, 4096 33, 16384 105).
__global__ void __launch_bounds__(kPagesThreads) __cluster_dims__(kPagesCluster, 1, 1)
    pages_reserve_kernel(const ReserveArgs a) {
  __shared__ WarpCounts s;
  wait_stream();
  const uint32_t rank = cluster_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = static_cast<int>(rank) * (kPagesThreads / 32) + warp;
  int64_t p0, p1;
  warp_share(a.P, g, p0, p1);
  const int per = (a.R + kPagesWarps - 1) / kPagesWarps;  // rows of a warp
  const int r0 = static_cast<int>(min(static_cast<int64_t>(a.R), static_cast<int64_t>(g) * per));
  const int r1 = static_cast<int>(min(static_cast<int64_t>(a.R), static_cast<int64_t>(r0) + per));
  int nfree = 0;
#pragma unroll 4
  for (int64_t p = p0 + lane; p < p1; p += 32) nfree += a.ref[p] <= 0 ? 1 : 0;
  nfree = __reduce_add_sync(0xffffffffu, nfree);
  int nneed = 0;
  for (int r = r0; r < r1; ++r) {
    int64_t b, e;
    int first, last;
    reserve_span(a, r, b, e, first, last);
    for (int j = first + lane; j <= last; j += 32)
      nneed += reserve_need(a, a.table[static_cast<int64_t>(r) * a.M + j]) != 0 ? 1 : 0;
  }
  nneed = __reduce_add_sync(0xffffffffu, nneed);
  int mine[2], total[2];
  scan_warp_counts(s, rank, nfree, nneed, mine, total);
  const int want = total[1];
  const bool fits = want <= total[0];
  if (rank == 0 && threadIdx.x == 0) a.lacking[0] = fits ? 0 : want - total[0];
  if (fits) {
    int k0 = mine[0];
    for (int64_t p = p0; p < p1 && k0 < want; p += 32) {
      const bool is = p + lane < p1 && a.ref[p + lane] <= 0;
      const uint32_t m = __ballot_sync(0xffffffffu, is);
      const int k = k0 + __popc(m & ((1u << lane) - 1u));
      if (is && k < want) a.fresh[k] = static_cast<int32_t>(p + lane);
      k0 += __popc(m);
    }
  }
  cluster_sync_all();
  int k0 = mine[1];
  for (int r = r0; r < r1; ++r) {
    int64_t b, e;
    int first, last;
    reserve_span(a, r, b, e, first, last);
    const int64_t in_page = (static_cast<int64_t>(1) << a.log_rows) - 1;
    const bool cut_head = (b & in_page) != 0, cut_tail = (e & in_page) != 0;
    int copy_from[2] = {-1, -1}, copy_to[2] = {-1, -1};
    for (int j0 = first; fits && j0 <= last; j0 += 32) {
      const int j = j0 + lane;
      int32_t* entry = a.table + static_cast<int64_t>(r) * a.M + j;
      const int p = j <= last ? *entry : 0;
      const int need = j <= last ? reserve_need(a, p) : 0;
      const uint32_t m = __ballot_sync(0xffffffffu, need != 0);
      if (need != 0) {
        const int k = k0 + __popc(m & ((1u << lane) - 1u));
        const int page = a.fresh[k];
        *entry = page;
        a.left[k] = need == 2 ? p : -1;
        if (need == 2) {  // its rows outside [begin, end) come along
          const int slot = j == first ? 0 : 1;
          if ((j == first && (cut_head || (first == last && cut_tail))) || (j == last && first != last && cut_tail)) {
            copy_from[slot] = p;
            copy_to[slot] = page;
          }
        }
      }
      k0 += __popc(m);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // at most one lane holds each (page ids are not negative)
      const int from = __reduce_max_sync(0xffffffffu, copy_from[i]);
      const int to = __reduce_max_sync(0xffffffffu, copy_to[i]);
      if (lane == i) {
        a.src[2 * static_cast<int64_t>(r) + i] = from;
        a.dst[2 * static_cast<int64_t>(r) + i] = to;
      }
    }
  }
  cluster_sync_all();
  if (!fits) return;
  for (int k = static_cast<int>(rank) * kPagesThreads + threadIdx.x; k < want; k += kPagesCluster * kPagesThreads) {
    a.ref[a.fresh[k]] = 1;
    const int p = a.left[k];
    if (p >= 0) atomicSub(a.ref + p, 1);
  }
}

// ---------------------------------------------------------------------------------------- compact

// With L live pages, the k-th live page at or above L moves to the k-th free page below L.  (1) count the
// live pages of each share; (2) the free pages below L and the live ones from L on; (3) their lists and
// the map of the pages that stay; (4) the map of those that move, and the counts; (5) a small table.
__global__ void __launch_bounds__(kPagesThreads) __cluster_dims__(kPagesCluster, 1, 1)
    pages_compact_kernel(const CompactArgs a) {
  __shared__ WarpCounts s;
  wait_stream();
  const uint32_t rank = cluster_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = static_cast<int>(rank) * (kPagesThreads / 32) + warp;
  const int gtid = static_cast<int>(rank) * kPagesThreads + threadIdx.x;
  int64_t p0, p1;
  warp_share(a.P, g, p0, p1);
  int live = 0;
#pragma unroll 4
  for (int64_t p = p0 + lane; p < p1; p += 32) live += a.ref[p] > 0 ? 1 : 0;
  live = __reduce_add_sync(0xffffffffu, live);
  int mine[2], total[2];
  scan_warp_counts(s, rank, live, 0, mine, total);
  const int L = total[0];
  int gaps = 0, moves = 0;
#pragma unroll 4
  for (int64_t p = p0 + lane; p < p1; p += 32) {
    const bool is = a.ref[p] > 0;
    gaps += !is && p < L ? 1 : 0;
    moves += is && p >= L ? 1 : 0;
  }
  gaps = __reduce_add_sync(0xffffffffu, gaps);
  moves = __reduce_add_sync(0xffffffffu, moves);
  cluster_sync_all();  // every CTA has read the first counts before they are replaced
  scan_warp_counts(s, rank, gaps, moves, mine, total);
  int kg = mine[0], km = mine[1];
  for (int64_t p = p0; p < p1; p += 32) {
    const int id = static_cast<int>(p) + lane;
    const bool in = id < p1;
    const bool is = in && a.ref[id] > 0;
    const bool gap = in && !is && id < L, move = is && id >= L;
    const uint32_t mg = __ballot_sync(0xffffffffu, gap), mm = __ballot_sync(0xffffffffu, move);
    const uint32_t below = (1u << lane) - 1u;
    if (gap) a.dst[kg + __popc(mg & below)] = id;
    if (move) a.src[km + __popc(mm & below)] = id;
    if (in && !move) a.remap[id] = is ? id : -1;
    if (in && !is) a.ref[id] = 0;
    kg += __popc(mg);
    km += __popc(mm);
  }
  const int n = total[0];  // = total[1]: as many gaps below L as live pages above
  for (int64_t k = n + static_cast<int64_t>(gtid); k < a.P / 2; k += kPagesCluster * kPagesThreads) a.src[k] = a.dst[k] = -1;
  if (gtid == 0) a.n_live[0] = L;
  cluster_sync_all();
  for (int k = gtid; k < n; k += kPagesCluster * kPagesThreads) {
    const int from = a.src[k], to = a.dst[k];
    a.remap[from] = to;
    a.ref[to] = a.ref[from];
    a.ref[from] = 0;
  }
  if (a.table == nullptr) return;
  cluster_sync_all();
  for (int i = gtid; i < a.entries; i += kPagesCluster * kPagesThreads) {
    const int p = a.table[i];
    a.table[i] = static_cast<unsigned>(p) < static_cast<unsigned>(a.P) ? a.remap[p] : -1;
  }
}

// table[i] = remap[table[i]] (no page where it names none): a large table, over all SMs.
__global__ void __launch_bounds__(256) pages_relabel_kernel(int32_t* table, int64_t n, int P,
                                                            const int32_t* remap) {
  wait_stream();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int p = table[i];
    table[i] = static_cast<unsigned>(p) < static_cast<unsigned>(P) ? remap[p] : -1;
  }
}

// ---------------------------------------------------------------------------------------- copy

// pages[dst[i]] = pages[src[i]] for every i whose two ids name pages.  A CTA takes pieces of kCopyPiece
// bytes of an entry in turn; each thread's loads of a piece are issued before its stores.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyPiece = kCopyThreads * kCopyUnroll * 16;

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(uint8_t* pages, int64_t page_bytes, int P,
                                                                  const int32_t* src,
                                                                  const int32_t* dst, int n, int pieces) {
  wait_stream();
  for (int64_t w = blockIdx.x; w < static_cast<int64_t>(n) * pieces; w += gridDim.x) {
    const int i = static_cast<int>(w / pieces);
    const int64_t at = (w % pieces) * static_cast<int64_t>(kCopyPiece) + threadIdx.x * 16;
    const int from = ld_after_wait(src + i), to = ld_after_wait(dst + i);
    if (static_cast<unsigned>(from) >= static_cast<unsigned>(P) || static_cast<unsigned>(to) >= static_cast<unsigned>(P) ||
        from == to)
      continue;
    const uint8_t* f = pages + from * page_bytes;
    uint8_t* t = pages + to * page_bytes;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (at + u * kCopyThreads * 16 < page_bytes) v[u] = *reinterpret_cast<const uint4*>(f + at + u * kCopyThreads * 16);
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (at + u * kCopyThreads * 16 < page_bytes) *reinterpret_cast<uint4*>(t + at + u * kCopyThreads * 16) = v[u];
  }
}

}  // namespace dsa
