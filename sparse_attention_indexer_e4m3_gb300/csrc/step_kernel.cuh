// A serving step's small calls over the paged bf16 cache: the tokens' maps from the sequences' lengths, packed keys to rows
// of the pages, and rows into their pages.
#pragma once

#include <climits>

#include "kv4.cuh"
#include "kv4_codec_kernel.cuh"
#include "paged.cuh"

namespace dsa {

// Row of the pages, seen as one matrix [P * page_rows], that row `pos` of sequence `seq` is; -1 where it has none.
__device__ __forceinline__ int64_t page_slot(const PageTable& c, int seq, int64_t pos) {
  if (static_cast<unsigned>(seq) >= static_cast<unsigned>(c.R) || pos < 0 || (pos >> c.log_rows) >= c.M) return -1;
  const int page = ld_after_wait(c.table + static_cast<int64_t>(seq) * c.M + (pos >> c.log_rows));
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.P)) return -1;
  return (static_cast<int64_t>(page) << c.log_rows) + (pos & ((1 << c.log_rows) - 1));
}

// ------------------------------------------------------------------------------------ the step's tokens

constexpr int kMapThreads = 256;
constexpr int kMapEach = 4;                          // sequences of a thread at a time
constexpr int kMapSeqs = kMapThreads * kMapEach;     // sequences scanned at a time
constexpr int kMapTokens = 1024;                     // tokens of a block

// With A_r = the sum of added[r'] and K_r that of held[r'] + added[r'] over r' < r, the tokens [A_r, A_r + added[r]) are
// sequence r's: token t is at position held[r] + t - A_r, its packed keys are [K_r, K_r + position].  A block takes
// 1024 tokens: it scans the lengths, 1024 sequences at a time, and each token of its share that falls among them finds
// its sequence by bisection.  All blocks scan from the first sequence on: no second launch, and even 65536 tokens of
// 4096 sequences are 64 blocks of four scans.  A launch's latency bounds it: with store_kv behind it 6.8 us for 64 rows.
__global__ void __launch_bounds__(kMapThreads) step_maps_kernel(const StepMapArgs a) {
  __shared__ int64_t at_s[kMapSeqs + 1];   // A_r of the sequences at hand, and behind the last
  __shared__ int64_t key_s[kMapSeqs];      // K_r
  __shared__ int held_s[kMapSeqs];
  __shared__ int64_t warp_s[2][kMapThreads / 32];
  wait_stream();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kMapTokens, t1 = min(t0 + kMapTokens, static_cast<int64_t>(a.T));
  int64_t tokens = 0, keys = 0;  // before the sequences at hand
  for (int64_t r0 = 0; r0 < a.R && tokens < t1; r0 += kMapSeqs) {
    int64_t add[kMapEach], both[kMapEach], sum_a = 0, sum_k = 0;
    int hold[kMapEach];
#pragma unroll
    for (int i = 0; i < kMapEach; ++i) {
      const int64_t r = r0 + threadIdx.x * kMapEach + i;
      hold[i] = r < a.R ? max(0, ld_after_wait(a.held + r)) : 0;
      add[i] = r < a.R ? max(0, ld_after_wait(a.added + r)) : 0;
      both[i] = hold[i] + add[i];
      sum_a += add[i];
      sum_k += both[i];
    }
    int64_t in_a = sum_a, in_k = sum_k;  // up to this thread, in its warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, in_a, o), y = __shfl_up_sync(0xffffffffu, in_k, o);
      if (lane >= o) {
        in_a += x;
        in_k += y;
      }
    }
    if (lane == 31) {
      warp_s[0][warp] = in_a;
      warp_s[1][warp] = in_k;
    }
    __syncthreads();
    int64_t before_a = tokens, before_k = keys;
#pragma unroll
    for (int w = 0; w < kMapThreads / 32; ++w) {
      if (w < warp) {
        before_a += warp_s[0][w];
        before_k += warp_s[1][w];
      }
      tokens += warp_s[0][w];
      keys += warp_s[1][w];
    }
    before_a += in_a - sum_a;
    before_k += in_k - sum_k;
    const int64_t from = tokens;  // (behind the sequences at hand)
#pragma unroll
    for (int i = 0; i < kMapEach; ++i) {
      const int s = threadIdx.x * kMapEach + i;
      at_s[s] = before_a;
      key_s[s] = before_k;
      held_s[s] = hold[i];
      before_a += add[i];
      before_k += both[i];
    }
    if (threadIdx.x == 0) at_s[kMapSeqs] = from;
    __syncthreads();
    for (int64_t t = max(t0, at_s[0]) + threadIdx.x; t < min(t1, from); t += kMapThreads) {
      int lo = 0, hi = kMapSeqs;  // at_s[lo] <= t < at_s[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at_s[mid] <= t)
          lo = mid;
        else
          hi = mid;
      }
      const int64_t pos = min(held_s[lo] + t - at_s[lo], static_cast<int64_t>(INT_MAX));
      a.seq[t] = static_cast<int>(r0) + lo;
      a.pos[t] = static_cast<int>(pos);
      a.ks[t] = static_cast<int>(min(key_s[lo], static_cast<int64_t>(INT_MAX)));
      a.ke[t] = static_cast<int>(min(key_s[lo] + pos + 1, static_cast<int64_t>(INT_MAX)));
    }
    __syncthreads();
  }
  for (int64_t t = max(t0, tokens) + threadIdx.x; t < t1; t += kMapThreads) {
    a.seq[t] = a.pos[t] = -1;
    a.ks[t] = a.ke[t] = 0;
  }
}

// ------------------------------------------------------------------------------------ packed keys to rows

constexpr int kSlotThreads = 256;
constexpr int kSlotEach = 4;  // entries of a thread at a time

// Entry v of token t names row v - start[t] of sequence seq[t].  A thread takes four entries of a row, in one access each where they
// are aligned; the table's entries come from L1 and L2.  A block takes a piece of some rows one after the other (no division by
// the pieces of a row: with one, lists of 8192 x 2048 took 31 us instead of 28 to 29).  Those 134 MB move at 4.6 to 4.8 TB/s, 70% of
// a copy's rate: 43 instructions an entry, in 64 bits, take some 19 us of it.  61 x 2048 entries take 3.6 us, a launch's latency.
__global__ void __launch_bounds__(kSlotThreads) page_slots_kernel(const PageTable c, const int32_t* seq, const int32_t* start,
                                                                  const int32_t* idx, int T, int K, int32_t* slots, bool wide) {
  wait_stream();
  const int64_t k = (static_cast<int64_t>(blockIdx.x) * kSlotThreads + threadIdx.x) * kSlotEach;
  if (k >= K) return;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    const int s = ld_after_wait(seq + t);
    const int64_t from = start != nullptr ? ld_after_wait(start + t) : 0;
    const int32_t* in = idx + t * K + k;
    int32_t* out = slots + t * K + k;
    int v[kSlotEach];
    if (wide) {
      const int4 w = ld_after_wait(reinterpret_cast<const int4*>(in));
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
#pragma unroll
      for (int j = 0; j < kSlotEach; ++j) v[j] = k + j < K ? ld_after_wait(in + j) : -1;
    }
#pragma unroll
    for (int j = 0; j < kSlotEach; ++j) v[j] = v[j] < 0 ? -1 : static_cast<int>(page_slot(c, s, v[j] - from));
    if (wide) {
      *reinterpret_cast<int4*>(out) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < kSlotEach; ++j)
        if (k + j < K) out[j] = v[j];
    }
  }
}

// ------------------------------------------------------------------------------------ rows into their pages

constexpr int kStoreThreads = 256;

// Row i of kv as row pos[i] of sequence seq[i], kBytes (32, or 16 where a row's place is not aligned to them) a thread; rows
// without a place are left out.  A copy, bound by memory: with step_maps before it 26 us for 65536 rows of 512 (5.2 TB/s of 134
// MB; by 16 bytes a thread 32 us).
template <int kBytes>
__global__ void __launch_bounds__(kStoreThreads) store_kv_kernel(const uint16_t* kv, int64_t stride, int N, int log_pieces,
                                                                 const int32_t* seq, const int32_t* pos, const int32_t* lacking,
                                                                 uint16_t* pages, const PageTable c) {
  wait_stream();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kStoreThreads + threadIdx.x;
  const int64_t row = i >> log_pieces;
  if (row >= N) return;
  if (lacking != nullptr && ld_after_wait(lacking) != 0) return;
  const int piece = static_cast<int>(i) & ((1 << log_pieces) - 1);
  const uint16_t* from = kv + row * stride + piece * (kBytes / 2);
  const int s = ld_after_wait(seq + row), at = ld_after_wait(pos + row);
  if constexpr (kBytes == 32) {
    uint32_t v[8];
    ld_32(from, v);
    const int64_t slot = page_slot(c, s, at);
    if (slot >= 0) st_32(pages + ((slot << log_pieces) + piece) * 16, v);
  } else {
    const uint4 v = ld_after_wait(reinterpret_cast<const uint4*>(from));
    const int64_t slot = page_slot(c, s, at);
    if (slot >= 0) reinterpret_cast<uint4*>(pages)[(slot << log_pieces) + piece] = v;
  }
}

}  // namespace dsa
