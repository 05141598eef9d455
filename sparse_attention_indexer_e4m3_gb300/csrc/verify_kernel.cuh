// Drafted tokens against the target's probabilities, with given random numbers (rejection sampling).  Row r drafted
// n = count[r] tokens d_i from probabilities q_i; p_i are the target's.  Token i is accepted while
// u_i q_i[d_i] < p_i[d_i], so with probability min(1, p / q); with a the number accepted before the first refusal, the token
// that follows is drawn from
//     w[v] = max(p_a[v] - q_a[v], 0)  where one was refused (p_a where that is all zero),   w = p_n  where none was:
// the lowest v with w[0] + ... + w[v] > u_G (w[0] + ... + w[V - 1]).  The accepted and the drawn token then follow the
// target's distribution.
//
// Sums in whole numbers: a probability is taken in units of 2^-56 (rounded to the nearest, so off by at most 2^-57), which
// sums exactly in 64 bits in any order, so the token does not depend on how the row is split.  What has less than
// 2^-57 is never drawn.  u S for a sum S of these units is compared by its whole part, which is exact, too.
//
// One cluster of CTAs a row, each with an equal share of the vocabulary.  All of them decide on the accepted ones (the
// few entries that takes are read by each); the sums of the shares are exchanged through the cluster's shared memory, and
// the warp into whose part the drawn number falls looks for the token: first among the sums that it kept of each
// piece of its part, then among that piece's values, which are in L2.
// It reads two rows of V floats a row, from the first access to the last in a chain of: counts and tokens,
// probabilities of the tokens, the rows, the exchange, one piece again.
#pragma once

#include "cluster.cuh"
#include "kv4.cuh"
#include "paged.cuh"

namespace dsa {

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerPiece = 128;      // values summed together, at least
constexpr int kVerPieces = 2048;    // most pieces of a CTA's share
constexpr int kVerMaxCluster = 8;

// A probability in units of 2^-56, nearest (0 where it is not above 0 or no number; above 1: 1).
__device__ __forceinline__ uint64_t prob_units(float p) {
  p = p > 0.f ? fminf(p, 1.f) : 0.f;
  const float a = p * 268435456.f;  // 2^28 (exact)
  const uint32_t hi = static_cast<uint32_t>(a);
  const uint32_t lo = __float2uint_rn((a - static_cast<float>(hi)) * 268435456.f);  // (the difference is exact; < 2^28)
  return (static_cast<uint64_t>(hi) << 28) + lo;
}

// u in [0, 1) in units of 2^-64 (what lies outside, or is no number, to the nearest in it or 0).
__device__ __forceinline__ uint64_t unit_fraction(float u) {
  if (!(u > 0.f)) return 0ull;
  if (u >= 1.f) return ~0ull;
  const float a = u * 4294967296.f;
  const uint32_t hi = static_cast<uint32_t>(a);
  const float rest = (a - static_cast<float>(hi)) * 4294967296.f;  // (a < 2^24 or a whole number: exact; < 2^32)
  return (static_cast<uint64_t>(hi) << 32) | static_cast<uint32_t>(rest);
}

__device__ __forceinline__ uint64_t warp_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kVerThreads) verify_drafts_kernel(const VerifyArgs a, int cluster, int piece, int pieces) {
  __shared__ uint64_t piece_s[kVerPieces];   // sums of this share's pieces
  __shared__ uint64_t warp_s[kVerWarps];
  __shared__ uint64_t share_s;               // of this share (read by the cluster)
  __shared__ int decide_s[2];                // accepted, whether one was refused
  wait_stream();
  const int rank = static_cast<int>(cluster_rank());
  const int r = static_cast<int>(blockIdx.x) / cluster;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t V = a.V;
  const int count = min(ld_after_wait(a.count + r), a.G);
  if (count < 0) {  // (the whole cluster)
    if (rank == 0 && threadIdx.x == 0) {
      a.accepted[r] = 0;
      a.token[r] = -1;
    }
    return;
  }
  const float* target = a.target + static_cast<int64_t>(r) * (a.G + 1) * V;
  const float* draft = a.draft + static_cast<int64_t>(r) * a.G * V;
  const float* u = a.u + static_cast<int64_t>(r) * (a.G + 1);
  if (warp == 0) {
    int n = 0;
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int i = i0 + lane;
      bool ok = false;
      if (i < count) {
        const int d = ld_after_wait(a.tokens + static_cast<int64_t>(r) * a.G + i);
        if (d >= 0 && d < a.V) {
          const float p = ld_after_wait(target + i * V + d), q = ld_after_wait(draft + i * V + d);
          ok = static_cast<double>(ld_after_wait(u + i)) * static_cast<double>(q) < static_cast<double>(p);  // (the product is exact)
        }
      }
      const uint32_t refused = __ballot_sync(0xffffffffu, i < count && !ok);
      if (refused != 0u) {
        n += __ffs(refused) - 1;
        break;
      }
      n += min(32, count - i0);
    }
    if (lane == 0) decide_s[0] = n;
  }
  __syncthreads();
  const int n = decide_s[0];
  const float* p_row = target + static_cast<int64_t>(n) * V;
  const uint64_t frac = unit_fraction(ld_after_wait(u + a.G));
  // this share's pieces, and this warp's among them
  const int64_t first = static_cast<int64_t>(pieces) * rank / cluster, last = static_cast<int64_t>(pieces) * (rank + 1) / cluster;
  const int w0 = static_cast<int>((last - first) * warp / kVerWarps), w1 = static_cast<int>((last - first) * (warp + 1) / kVerWarps);
  // the second time only where nothing is left of the target over the draft
  for (int attempt = 0; attempt < 2; ++attempt) {
    const float* q_row = n < count && attempt == 0 ? draft + static_cast<int64_t>(n) * V : nullptr;
    const auto weight = [&](int64_t v) -> uint64_t {
      const uint64_t p = prob_units(ld_after_wait(p_row + v));
      if (q_row == nullptr) return p;
      const uint64_t q = prob_units(ld_after_wait(q_row + v));
      return p > q ? p - q : 0ull;
    };
    uint64_t mine = 0;
    for (int i = w0; i < w1; ++i) {
      const int64_t v0 = (first + i) * piece, v1 = min(v0 + piece, V);
      uint64_t sum = 0;
      for (int64_t v = v0 + lane; v < v1; v += kVerPiece) {
        float p[4], q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool in = v + 32 * k < v1;
          p[k] = in ? ld_after_wait(p_row + v + 32 * k) : 0.f;
          q[k] = in && q_row != nullptr ? ld_after_wait(q_row + v + 32 * k) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t x = prob_units(p[k]), y = prob_units(q[k]);
          sum += x > y ? x - y : 0ull;
        }
      }
      sum = warp_sum_u64(sum);
      if (lane == 0) piece_s[i] = sum;
      mine += sum;
    }
    if (lane == 0) warp_s[warp] = mine;
    __syncthreads();
    uint64_t before = 0, share = 0;  // of the warps before, of this share
#pragma unroll
    for (int w = 0; w < kVerWarps; ++w) {
      if (w < warp) before += warp_s[w];
      share += warp_s[w];
    }
    if (threadIdx.x == 0) share_s = share;
    cluster_sync_all();
    uint64_t all = 0;
    for (int k = 0; k < cluster; ++k) {
      const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&share_s));
      const uint64_t x = static_cast<uint32_t>(ld_cluster_s32(at, k)) | (static_cast<uint64_t>(static_cast<uint32_t>(ld_cluster_s32(at + 4, k))) << 32);
      if (k < rank) before += x;
      all += x;
    }
    cluster_sync_all();  // (share_s is written anew, or the CTA ends)
    if (all == 0ull) {
      if (q_row != nullptr) continue;
      if (rank == 0 && threadIdx.x == 0) {  // a target without a probability
        a.accepted[r] = n;
        a.token[r] = -1;
      }
      return;
    }
    const uint64_t drawn = __umul64hi(frac, all);  // floor(u S) < S
    if (drawn < before || drawn - before >= mine) return;
    // the piece, then the value
    uint64_t left = drawn - before;
    int i = w0;
    for (; i < w1 - 1 && left >= piece_s[i]; ++i) left -= piece_s[i];
    const int64_t v0 = (first + i) * piece, v1 = min(v0 + piece, V);
    for (int64_t v = v0; v < v1; v += 32) {
      const uint64_t x = v + lane < v1 ? weight(v + lane) : 0ull;
      uint64_t s = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, s > left);
      if (past != 0u) {
        if (lane == 0) {
          a.accepted[r] = n;
          a.token[r] = static_cast<int>(v + __ffs(past) - 1);
        }
        return;
      }
      left -= __shfl_sync(0xffffffffu, s, 31);
    }
    return;
  }
}

}  // namespace dsa
