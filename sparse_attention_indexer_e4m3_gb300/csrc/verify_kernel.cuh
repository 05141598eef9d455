// Drafted tokens against the target's probabilities, with given random numbers (rejection sampling).  Row r drafted
// n = count[r] tokens d_i from probabilities q_i; p_i are the target's.  Token i is accepted while
// u_i q_i[d_i] < p_i[d_i], so with probability min(1, p / q); with a the number accepted before the first refusal, the token
// that follows is drawn from
//     w[v] = max(p_a[v] - q_a[v], 0)  where one was refused (p_a where that is all zero),   w = p_n  where none was:
// the lowest v with w[0] + ... + w[v] > u_G (w[0] + ... + w[V - 1]).  The accepted and the drawn token then follow the
// target's distribution.
//
// Sums in whole numbers: a probability is taken in units of 2^-55, rounded to the nearest (what is 2^-32 or more is not rounded
// at all), which sums exactly in 64 bits in any order, so the token does not depend on how the row is split.  What has less than
// 2^-56 is never drawn.  u S for a sum S of these units is compared by its whole part, which is exact, too.
//
// One cluster of CTAs a row, each with an equal share of the vocabulary.  All of them decide on the accepted ones (the
// few entries that takes are read by each); the sums of the shares are exchanged through the cluster's shared memory, and
// the warp into whose part the drawn number falls looks for the token: first among the sums that it kept of each
// piece of its part, then among that piece's values, which are in L2.
// It reads two rows of V floats a row, in a chain of: counts and tokens, probabilities of the tokens, the rows, the
// exchange, one piece again.  A row of 131072 takes 10.3 us (a launch and that chain: its bytes take 0.2), 128 rows of 50257
// 21.4 us, 2.4 TB/s: the sums' additions, 55 instructions a pair of values on all SMs, take about half of it (13.6 million
// instructions of warps, some 11 us) and the chain the rest.
// Three pieces at once a warp with 64 registers and two CTAs an SM: 21.4 us; one piece, 32 registers and four CTAs: 23.5.
#pragma once

#include "cluster.cuh"
#include "kv4.cuh"
#include "paged.cuh"

namespace dsa {

constexpr int kVerThreads = 512;    // two CTAs an SM; where the rows leave SMs without work one of kVerMostThreads (a row 10.3 us for 12.1)
constexpr int kVerMostThreads = 1024;
constexpr int kVerPiece = 128;      // values summed together, at least
constexpr int kVerPieces = 2048;    // most pieces of a CTA's share
constexpr int kVerMaxCluster = 8;

// Weights max(p - q, 0) in units of 2^-55 (what is no number or below 0 counts as 0, above 1 as 1), summed.  A probability x in [0, 1]
// is rounded to a multiple of 2^-22 by adding 3, whose neighbours are 2^-22 apart, so that the sum's bits are 3's and that multiple;
// what is left is exact, and rounded likewise to a multiple of 2^-44, and what is left of that to one of 2^-55.  Eight additions a
// value, all but the bits' in fp32.  128 rows of 50257 took 23.5 us with them, 27.8 with conversions to whole numbers and
// 24.5 with shifts of the mantissa.
struct WeightSum {
  int part[3] = {0, 0, 0};  // of up to 2^8 weights, in units of 2^-22, 2^-44 and 2^-55

  __device__ __forceinline__ void add(float p, float q) {
    p = fminf(fmaxf(p, 0.f), 1.f);
    q = fminf(fmaxf(q, 0.f), p);
    const float at[3] = {3.f, 1.5f / (1 << 21), 1.5f / (1ull << 32)};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const float x = __fadd_rn(p, at[i]), y = __fadd_rn(q, at[i]);
      part[i] += __float_as_int(x) - __float_as_int(y);
      p = __fsub_rn(p, __fsub_rn(x, at[i]));
      q = __fsub_rn(q, __fsub_rn(y, at[i]));
    }
  }
  __device__ __forceinline__ uint64_t units() const {
    return static_cast<uint64_t>((static_cast<int64_t>(part[0]) << 33) + (static_cast<int64_t>(part[1]) << 11) + part[2]);
  }
};

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

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) verify_drafts_kernel(const VerifyArgs a, int cluster, int piece, int pieces) {
  __shared__ uint64_t piece_s[kVerPieces];                 // sums of this share's pieces
  constexpr int warps = kThreads / 32;
  __shared__ uint64_t warp_s[warps];
  __shared__ uint64_t share_s[2][kVerMaxCluster];          // by attempt: of the cluster's shares, written by each of them
  __shared__ int decide_s;                                 // accepted
  wait_stream();
  cluster_arrive();
  const int rank = static_cast<int>(cluster_rank());
  const int r = static_cast<int>(blockIdx.x) / cluster;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t V = a.V;
  const float* target = a.target + static_cast<int64_t>(r) * (a.G + 1) * V;
  const float* draft = a.draft + static_cast<int64_t>(r) * a.G * V;
  const float* u = a.u + static_cast<int64_t>(r) * (a.G + 1);
  const uint64_t frac = unit_fraction(ld_after_wait(u + a.G));
  // (the first tokens and their numbers are read beside the count)
  int d = -1;
  float mine_u = 0.f;
  const auto draft_of = [&](int i) {
    d = i < a.G ? ld_after_wait(a.tokens + static_cast<int64_t>(r) * a.G + i) : -1;
    mine_u = i < a.G ? ld_after_wait(u + i) : 0.f;
  };
  if (warp == 0) draft_of(lane);
  const int count = min(ld_after_wait(a.count + r), a.G);
  if (count < 0) {  // (the whole cluster)
    cluster_wait();
    if (rank == 0 && threadIdx.x == 0) {
      a.accepted[r] = 0;
      a.token[r] = -1;
    }
    return;
  }
  if (warp == 0) {
    int n = 0;
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int i = i0 + lane;
      if (i0 > 0) draft_of(i);
      bool ok = false;
      if (i < count && d >= 0 && d < a.V) {
        const float p = ld_after_wait(target + i * V + d), q = ld_after_wait(draft + i * V + d);
        ok = static_cast<double>(mine_u) * static_cast<double>(q) < static_cast<double>(p);  // (the product is exact)
      }
      const uint32_t refused = __ballot_sync(0xffffffffu, i < count && !ok);
      if (refused != 0u) {
        n += __ffs(refused) - 1;
        break;
      }
      n += min(32, count - i0);
    }
    if (lane == 0) decide_s = n;
  }
  __syncthreads();
  const int n = decide_s;
  if (rank == 0 && threadIdx.x == 0) {  // (the warp that finds the token writes it, behind the exchange)
    a.accepted[r] = n;
    a.token[r] = -1;
  }
  const float* p_row = target + static_cast<int64_t>(n) * V;
  // this share's pieces, and this warp's among them
  const int64_t first = static_cast<int64_t>(pieces) * rank / cluster, last = static_cast<int64_t>(pieces) * (rank + 1) / cluster;
  const int w0 = static_cast<int>((last - first) * warp / warps), w1 = static_cast<int>((last - first) * (warp + 1) / warps);
  // the second time only where nothing is left of the target over the draft
  for (int attempt = 0; attempt < 2; ++attempt) {
    const float* q_row = n < count && attempt == 0 ? draft + static_cast<int64_t>(n) * V : nullptr;
    // the sums of its pieces, some at a time for loads in flight (one in the larger CTAs, whose warps have four of them at V = 131072 and
    // one or two up to 65536)
    constexpr int kAhead = kThreads == kVerThreads ? 3 : 1;
    uint64_t mine = 0;
    for (int i = w0; i < w1; i += kAhead) {
      uint64_t sum[kAhead];
#pragma unroll
      for (int h = 0; h < kAhead; ++h) sum[h] = 0;
      const int64_t v0 = (first + i) * piece, end = min((first + min(i + kAhead, w1)) * piece, V);
      for (int64_t o = lane; o < piece; o += kVerPiece) {
        float p[kAhead][4], q[kAhead][4];
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int64_t at = v0 + h * static_cast<int64_t>(piece) + o + 32 * k;
            p[h][k] = at < end ? ld_after_wait(p_row + at) : 0.f;
            q[h][k] = at < end && q_row != nullptr ? ld_after_wait(q_row + at) : 0.f;
          }
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
          WeightSum w;
#pragma unroll
          for (int k = 0; k < 4; ++k) w.add(p[h][k], q[h][k]);
          sum[h] += w.units();
        }
      }
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        sum[h] = warp_sum_u64(sum[h]);
        if (lane == 0 && i + h < w1) piece_s[i + h] = sum[h];
        mine += sum[h];
      }
    }
    if (lane == 0) warp_s[warp] = mine;
    __syncthreads();
    uint64_t before = 0, share = 0;  // of the warps before, of this share
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += warp_s[w];
      share += warp_s[w];
    }
    if (attempt == 0) cluster_wait();  // (all CTAs of the cluster are there)
    // its sum to every CTA of the cluster (whose shared memory nobody reaches into behind the barrier)
    if (static_cast<int>(threadIdx.x) < cluster) st_cluster_u64(&share_s[attempt][rank], threadIdx.x, share);
    cluster_sync_all();
    uint64_t all = 0;
    for (int k = 0; k < cluster; ++k) {
      const uint64_t x = share_s[attempt][k];
      if (k < rank) before += x;
      all += x;
    }
    if (all == 0ull) {
      if (q_row != nullptr) continue;
      return;  // a target without a probability
    }
    const uint64_t drawn = __umul64hi(frac, all);  // floor(u S) < S
    if (drawn < before || drawn - before >= mine) return;
    // the piece, then the value
    uint64_t left = drawn - before;
    int i = w0;
    for (; i < w1 - 1 && left >= piece_s[i]; ++i) left -= piece_s[i];
    const int64_t v0 = (first + i) * piece, v1 = min(v0 + piece, V);
    for (int64_t v = v0; v < v1; v += kVerPiece) {
      uint64_t x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t at = v + 32 * k + lane;
        const float p = at < v1 ? ld_after_wait(p_row + at) : 0.f, q = at < v1 && q_row != nullptr ? ld_after_wait(q_row + at) : 0.f;
        WeightSum w;
        w.add(p, q);
        x[k] = w.units();
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint64_t s = x[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, s > left);
        if (past != 0u) {
          if (lane == 0) a.token[r] = static_cast<int>(v + 32 * k + __ffs(past) - 1);
          return;
        }
        left -= __shfl_sync(0xffffffffu, s, 31);
      }
    }
    return;
  }
}

}  // namespace dsa
