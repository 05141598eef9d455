// Sparse attention over the 4-bit paged cache on the tensor cores.  For query token t and head h, over
// the entries of idx[t, :] that name a mapped row j of the token's sequence (kv_j = r_j * v_j, v_j the
// exact fp16 values s * c of kv4.cuh):
//     x_j = scale * q[t,h,:] . kv_j
//     out[t,h,:] = sum_j e^{x_j} kv_j / ( sum_j e^{x_j} + e^{sink[h]} )
// Both products run on fp16 operands with fp32 accumulators.  v_j is exact; q is bf16 and becomes fp16 times a
// power of two of its head, each value off by at most 2^-23 of the head's largest (those down to 2^-15 of it not at all);
// the weights enter the second product as w_j = r_j * 2^(y_j - m), y = x log2 e,
// rounded to fp16 (half a step, 2^-11), with m a bound on y_j + log2 r_j so that w_j <= 2^8 whatever the
// row scales are.  fp16 weights rather than bf16 ones because their rounding would otherwise be as large as the
// output's own.
// The denominator is the sum of 2^(y_j - m) in fp32.  Its terms are w_j / r_j, without a second exponential, as long
// as none is lost where w_j underflows: m is at most (the largest y) + log2 of (the largest row scale so far), so with row
// scales within 2^100 of one another a row whose w_j is below 2^-126 has a weight below 2^-26 of the largest.  A
// block with row scales further below the largest so far (rows of zeros, held with r = 2^-100, beside rows of 2^11
// or more) forms its terms by an exponential of their own, which may be subnormal: y_j - m lies between -117 (for the largest
// y, as m is at most 117 above it) and 108 (rows of the least scale, 2^8 above the bound), so the largest keep 24 bits and
// more, and sums of up to 2^19 rows, 2^26 with scores that do not grow, do not overflow.
//
// A unit is (token, group of up to 64 heads, share of the token's list); a cluster of S CTAs shares
// one list and joins its S partial results, so a call with few tokens still uses most SMs and needs no second
// launch.  One CTA per SM, 896 threads, per block of 128 entries:
//   scout    (warps 1-3)   find the unit's blocks and, up to six blocks ahead, its entries' pages and row scales;
//   convert  (warps 20-27) the rows' codes to fp16 values, as D / 64 chunks of [128 keys x 128 bytes], 128-byte
//                          swizzled; a masked entry becomes a row of zeros (its memory is not read); and the
//                          unit's q to fp16;
//   score    (warp 0)      S^T = V . Q^T: M = 128 keys, N = 64 heads, K = D (tcgen05.mma kind::f16);
//   softmax  (warps 4-19)  thread = (key, 16 heads): weights as fp16 rows P[key][head]; the running
//                          bound m moves only when exceeded by more than 2^8;
//   weighted (warp 0)      O^T += V^T . P^T: M = 128 output dims (D / 128 tiles), N = 64, K = 128 keys.
// A tile of 128 dims is converted anew as soon as the weighted sum has read it; the global loads of the next
// block are in flight while its tiles are waited for.  Up to D = 256 two or four blocks fit, and the score product
// of the next block is issued before the weighted sum of the last, so the softmax runs beside it.
//
// What bounds it (D = 512, 64 heads, lists of 2048; 4096 tokens in 1.22 ms, 901 TFLOP/s, 47% of the measured
// bf16 rate; the attention over bf16 rows reaches 595 TFLOP/s): a tensor-core instruction of these shapes takes 52 to 63
// cycles whatever its 64 heads need (at 128 columns it does twice the work in 64), so a block's 64 instructions take
// 3,650 cycles of its 4,800; the softmax (1,500) stands between the two products, because one block and
// the 64 KB of q fill shared memory, and overlaps them in part.  At D = 256 and below a block takes 1.04 us (D = 64 and
// 128) to 1.34 us (256), the softmax's latency, against 2.6 at 512.  A unit costs 5,000 to 12,000 cycles beside its
// blocks (its q, its first block's way in, its output).  72 registers a thread are all that 896 threads have: the roles
// spill up to 28 bytes, and a change in one of them moves the others' time by a few percent.  Tried without gain: 8 softmax warps of 32 heads (registers), the next q brought
// by the softmax warps or by asynchronous copies, two buffers of P, register shares moved between the roles.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "attn_tc_kernel.cuh"
#include "cluster.cuh"
#include "kv4.cuh"
#include "launch.h"

namespace dsa {

// Row scales outside this range are clamped (the quantiser writes 2^-100 to 2^117).
constexpr float kKv4MinScale = 7.888609052210118e-31f;  // 2^-100

constexpr int kKv4SoftHeads = 16;         // heads of a softmax thread
constexpr int kKv4SoftThreads = kTcAttnKeys * kTcAttnHeads / kKv4SoftHeads;
constexpr int kKv4SoftWarps = kKv4SoftThreads / 32;
constexpr int kKv4FirstConv = 4 + kKv4SoftWarps;  // warps 0-3 issue and scout, then softmax, then convert
constexpr int kKv4ConvThreads = 256;
constexpr int kKv4ConvWarps = kKv4ConvThreads / 32;
constexpr int kKv4Threads = 32 * (kKv4FirstConv + kKv4ConvWarps);
constexpr int kKv4Scouts = 3;             // scout warps; one of them looks up every third block
constexpr int kKv4Slots = 2 * kKv4Scouts; // blocks whose entries are looked up ahead (a slot is always one scout's)
constexpr int kKv4Shares = kKv4MaxShares; // most CTAs that share a list
constexpr float kKv4NoBound = -3e38f;     // bound of a head without keys so far (finite: a masked key is minus infinity)
// q enters times 2^kKv4QExp where the largest value of its head has an exponent in [kKv4QLow, kKv4QHigh] (ordinary q), else
// times a power of two of the head, which brings that to [2^13, 2^14); the softmax then takes the unit's scores to one
// scale first (7% of a 4096-token prompt, 17% at D = 128).  In fp16 a value of 2^-17 or more is exact and others are
// off by at most 2^-25: here 2^-15 and 2^-23 of the head's largest.
constexpr int kKv4QExp = 7, kKv4QLow = -9, kKv4QHigh = 8;
constexpr float kKv4Spread = 1.2676506002282294e30f;  // 2^100: row scales within it share the weights' exponentials

template <int D>
struct AttnKv4Layout {
  static constexpr int kStages = D <= 128 ? 4 : (D <= 256 ? 2 : 1);  // kv blocks held
  static constexpr int kScores = kStages < 2 ? 1 : 2;           // score accumulators
  static constexpr int kChunks = D / 64;                        // chunks of a row in the score product
  static constexpr int kTiles = D >= 128 ? D / 128 : 1;         // output tiles (D = 64: half of one is zero)
  static constexpr int kTileWarps = kTiles > 1 ? kKv4ConvWarps / 2 : kKv4ConvWarps;  // warps that convert a tile
  static constexpr int kChunkBytes = kTcAttnKeys * 128;
  static constexpr int kStageBytes = 2 * kTiles * kChunkBytes;
  static constexpr int kQChunkBytes = kTcAttnHeads * 128;
  static constexpr int kKv = 0;
  static constexpr int kQ = kKv + kStages * kStageBytes;
  static constexpr int kP = kQ + kChunks * kQChunkBytes;        // fp16 [128 keys][64 heads]
  static constexpr int kEnt = kP + kTcAttnKeys * 128;           // int2 [slots][128]: page, row in the page
  static constexpr int kScl = kEnt + kKv4Slots * kTcAttnKeys * 8;  // float [slots][128]: row scale, 0 = masked
  static constexpr int kRed = kScl + kKv4Slots * kTcAttnKeys * 4;  // float [4][64] cross-warp scratch
  static constexpr int kMax = kRed + 4 * kTcAttnHeads * 4;      // float [64] running bound (log2 units)
  static constexpr int kAlpha = kMax + kTcAttnHeads * 4;        // float [64] rescale / output factors
  static constexpr int kJoin = kAlpha + kTcAttnHeads * 4;       // float [shares][64] factors of the shares
  static constexpr int kMisc = kJoin + kKv4Shares * kTcAttnHeads * 4;  // int [32]
  static constexpr int kQFac = kMisc + 128;                     // float [2][64] by unit: what undoes the heads' q factors
  static constexpr int kPhase = kQFac + 2 * kTcAttnHeads * 4;   // int [softmax warps]
  static constexpr int kBar = kPhase + kKv4SoftWarps * 4;
  static constexpr int kNumBars = 16 + 3 * kKv4Slots + 2 * kStages * kTiles;
  static constexpr int kSmem = kBar + kNumBars * 8 + 1024;      // + alignment slack
  // tensor memory: S^T (kScores of them) from column 0, O^T tile m from column 64 (kScores + m)
  static constexpr int kTmemCols = kScores + kTiles <= 4 ? 256 : 512;
};

// Instruction descriptor, kind::f16 with fp16 operands and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// One thread of the (converged) warp: 1 there, 0 elsewhere.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// tcgen05.mma kind::f16 and commit, issued where `on` is set.  The whole warp runs the issue loop, so that
// addresses and descriptors stay warp-uniform; a loop that one thread runs alone took 80 to 120 cycles per
// product instead of the tensor core's 52 to 63.
template <bool kAcc>
__device__ __forceinline__ void mma_f16_if(uint32_t on, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc = 1u) {
  if constexpr (kAcc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, 1, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(on)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(on), "r"(acc)
        : "memory");
  }
}
__device__ __forceinline__ void mma_commit_if(uint32_t on, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(on)
      : "memory");
}

// Two fp32 lanes in one register pair.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Reduces 16 values per lane (one of each of 16 heads) across the warp's 32 lanes, by recursive halving:
// afterwards v[0] holds head lane / 2.
template <class Op>
__device__ __forceinline__ void xpose_reduce16(float (&v)[16], int lane, Op op) {
#pragma unroll
  for (int half = 8, off = 16; half >= 1; half >>= 1, off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < half) {
        const float send = up ? v[i] : v[i + half];
        const float keep = up ? v[i + half] : v[i];
        v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
      }
    }
  }
  v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// 2^x, subnormal results included.
__device__ __forceinline__ float exp2_gradual(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Output factor of a head whose weights' bound is m (log2 units) and whose denominator, in units of
// 2^m, is l without the sink; writes the natural log of the whole denominator where lse is given.  0 for
// a head without keys (m = kKv4NoBound) and sink.  The larger of bound and sink is the unit, so neither overflows.
__device__ __forceinline__ float softmax_factor(float m, float l, const float* sink, int h, float* lse) {
  const bool keys = m != kKv4NoBound;
  float f = keys ? 1.f : 0.f, unit = m;
  if (!keys) l = 0.f;
  if (sink != nullptr) {
    const float s2 = ld_after_wait(sink + h) * 1.4426950408889634f;
    if (keys && s2 - m <= 64.f) {
      l += exp2f(s2 - m);
    } else if (s2 != -INFINITY) {
      if (keys) f = exp2f(m - s2);
      l = fmaf(l, f, 1.f);
      unit = s2;
    }
  }
  if (lse != nullptr) *lse = l > 0.f ? (unit + log2f(l)) * 0.6931471805599453f : -INFINITY;
  return l > 0.f ? f / l : 0.f;
}

// The larger magnitudes of two pairs of bf16 values (their signs mean nothing).
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two bf16 values to fp16, times f.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float f) {
  const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// kSingle: one unit per cluster, whose CTAs may share its list; else one CTA per unit, walking over the units.
template <int D, bool kSingle>
__global__ void __launch_bounds__(kKv4Threads, 1) sparse_attn_kv4_kernel(const AttnKv4Params p, int shares,
                                                                         unsigned* err) {
  using L = AttnKv4Layout<D>;
  constexpr int kCh = L::kChunks;
  constexpr int kTi = L::kTiles;
  constexpr int kSt = L::kStages;
  constexpr int kSc = L::kScores;
  extern __shared__ __align__(1024) uint8_t kv4_attn_smem[];
  uint8_t* smem = kv4_attn_smem + ((1024u - (smem_addr(kv4_attn_smem) & 1023u)) & 1023u);
  uint8_t* kv_s = smem + L::kKv;
  uint8_t* q_s = smem + L::kQ;
  uint8_t* p_s = smem + L::kP;
  int2* ent_s = reinterpret_cast<int2*>(smem + L::kEnt);
  float* scl_s = reinterpret_cast<float*>(smem + L::kScl);
  float* red_s = reinterpret_cast<float*>(smem + L::kRed);
  float* max_s = reinterpret_cast<float*>(smem + L::kMax);
  float* alpha_s = reinterpret_cast<float*>(smem + L::kAlpha);
  float* join_s = reinterpret_cast<float*>(smem + L::kJoin);
  // [0, 1] blocks of the units in flight, [16..18] by block modulo 3: a bound has to be raised, [20..31] by slot: its
  // smallest and largest row scale
  volatile int* misc = reinterpret_cast<volatile int*>(smem + L::kMisc);
  float* qfac_s = reinterpret_cast<float*>(smem + L::kQFac);
  float2* span_s = reinterpret_cast<float2*>(smem + L::kMisc + 80);
  static_assert(kKv4Slots <= 6, "spans of the slots lie behind the flags");
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  // (a barrier that its waiters may lag behind by more than a phase is a pair, or one per stage)
  uint64_t* q_full = bars + 0;  // [2]
  uint64_t* q_empty = bars + 2;
  uint64_t* p_full = bars + 3;
  uint64_t* pv_done = bars + 4;
  uint64_t* o_empty = bars + 5;
  uint64_t* unit_full = bars + 6;   // [2]
  uint64_t* unit_empty = bars + 8;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 10);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* drain = bars + 11;
  uint64_t* s_full = bars + 12;  // [score accumulator]
  uint64_t* checked = bars + 14;
  uint64_t* ent_full = bars + 15;
  uint64_t* scl_full = ent_full + kKv4Slots;
  uint64_t* ent_empty = scl_full + kKv4Slots;
  uint64_t* kv_full = ent_empty + kKv4Slots;  // [stage][tile]
  uint64_t* kv_empty = kv_full + kSt * kTi;
  uint64_t* soft_all = kv_empty + kSt * kTi;  // all softmax warps
  volatile uint32_t* phase_s = reinterpret_cast<volatile uint32_t*>(smem + L::kPhase);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int H = p.H;
  const int units = p.T * p.groups;
  const int share = kSingle ? static_cast<int>(blockIdx.x) % shares : 0;
  const int unit0 = kSingle ? static_cast<int>(blockIdx.x) / shares : static_cast<int>(blockIdx.x);
  const int unit_step = static_cast<int>(gridDim.x);

  if constexpr (D == 64) {  // the upper half of a 64-dim row's tile stays zero
    for (int s = 0; s < kSt; ++s)
      for (int i = threadIdx.x; i < L::kChunkBytes / 16; i += kKv4Threads)
        reinterpret_cast<uint4*>(kv_s + s * L::kStageBytes + L::kChunkBytes)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (threadIdx.x < 32) misc[threadIdx.x] = 0;
  if (threadIdx.x < kKv4SoftWarps) phase_s[threadIdx.x] = 0u;
  for (int i = threadIdx.x; i < kKv4Slots * kTcAttnKeys; i += kKv4Threads) ent_s[i] = make_int2(-1, 0);
  if (threadIdx.x == 0) {
    mbar_init(q_empty, 1);
    mbar_init(checked, kKv4SoftWarps);
    mbar_init(soft_all, kKv4SoftWarps);
    mbar_init(p_full, kKv4SoftWarps);
    mbar_init(pv_done, 1);
    mbar_init(o_empty, kKv4SoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], kKv4ConvWarps);
      mbar_init(&s_full[i], 1);
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_empty[i], 1 + kKv4SoftWarps + kKv4ConvWarps);
    }
    for (int i = 0; i < kKv4Slots; ++i) {
      mbar_init(&ent_full[i], 32);
      mbar_init(&scl_full[i], 32);
      mbar_init(&ent_empty[i], kKv4SoftWarps + kKv4ConvWarps);
    }
    for (int i = 0; i < kSt * kTi; ++i) {
      mbar_init(&kv_full[i], L::kTileWarps);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  fence_proxy_async_shared();
  // The set-up above overlaps the end of the kernel before.  Tensor memory is taken only after it: a kernel that lets its
  // dependents start early may still have to allocate its own, on an SM where this one would hold all of it and wait.
  wait_stream();
  if (warp == 0) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const uint32_t s_tmem = tbase;
  const uint32_t o_tmem = tbase + 64 * L::kScores;
  // this CTA's blocks of a unit whose list has `all` of them
  const auto first_block = [&](int all, int s) { return kSingle ? static_cast<int>(static_cast<int64_t>(all) * s / shares) : all * s; };
  const int rows = 1 << p.pool.log_rows;
  const int64_t page_bytes = static_cast<int64_t>(rows) * kv4_row_bytes(D);

  // A wait that expires, in any role, sets the abort flag, and later waits return at once; what happens then is bounded too:
  //   - a block count is used by a warp whose lanes all waited for it with success (gone() is the same for the whole
  //     warp, and true wherever a wait of one of its lanes failed), by the softmax warps if all of them did;
  //   - a page id is one that was found mapped, or -1 as from the start, whether the wait for it succeeded or not;
  //   - the softmax warps pass the same hardware barriers (whose wait has no limit): those of a unit and its first block, which
  //     they enter together or not at all.  Where they may differ on whether a bound has to be raised they meet at an
  //     mbarrier, in a bounded wait, and a warp may leave the blocks after the first at any time.
  const auto gone = [&]() -> bool { return __any_sync(0xffffffffu, *abort_flag != 0) != 0; };
  constexpr int kLook = 16;  // blocks between two looks at the abort flag

  // q of unit n (token t, heads [h0, h0 + nh)) as fp16 times a power of two of each head, by eight warps (w of them); the
  // place is written after free() returns true.  A warp takes whole heads, so the largest value of a head is known from
  // its own loads.
  const auto bring_q = [&](int w, int n, int t, int h0, int nh, auto free) -> bool {
    const uint16_t* q = p.q + (static_cast<int64_t>(t) * H + h0) * D;
    constexpr int kAcross = D / 8 < 32 ? D / 8 : 32;  // lanes of a head
    constexpr int kEach = D / 8 / kAcross;            // 16-byte pieces of a lane
    constexpr int kHeads = 32 / kAcross;              // heads at a time
    constexpr int kSteps = kTcAttnHeads / (kKv4ConvWarps * kHeads);
    constexpr int kMost = (D == 512 ? 8 : 4) / kEach;  // in flight at a time
    constexpr int kBatch = kSteps < kMost ? kSteps : kMost;
    const int head = w * kHeads + lane / kAcross, piece = lane % kAcross;
#pragma unroll 1
    for (int s0 = 0; s0 < kSteps; s0 += kBatch) {
      uint4 v[kBatch][kEach];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = (s0 + i) * kKv4ConvWarps * kHeads + head;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          v[i][k] = make_uint4(0u, 0u, 0u, 0u);
          if (h < nh) v[i][k] = ld_after_wait(reinterpret_cast<const uint4*>(q + static_cast<int64_t>(h) * D) + piece + kAcross * k);
        }
      }
      if (s0 == 0 && !free()) return false;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = (s0 + i) * kKv4ConvWarps * kHeads + head;
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          top = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(top, v[i][k].x), v[i][k].y), v[i][k].z), v[i][k].w);
        top = max(top & 0x7FFFu, (top >> 16) & 0x7FFFu);
#pragma unroll
        for (int o = kAcross / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = static_cast<int>(top >> 7) - 127;  // exponent of the largest
        int up = kKv4QExp;
        if (top != 0u && e < 128 && (e < kKv4QLow || e > kKv4QHigh)) up = min(13 - e, 126);  // it lands in [2^13, 2^14)
        const float f = __int_as_float((127 + up) << 23);
        if (piece == 0) qfac_s[(n & 1) * kTcAttnHeads + h] = __int_as_float((127 - up) << 23);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          const int pc = piece + kAcross * k;
          *reinterpret_cast<uint4*>(q_s + (pc / 8) * L::kQChunkBytes + swz128(h, (pc % 8) * 16)) =
              make_uint4(bf16x2_to_f16x2(v[i][k].x, f), bf16x2_to_f16x2(v[i][k].y, f), bf16x2_to_f16x2(v[i][k].z, f),
                         bf16x2_to_f16x2(v[i][k].w, f));
        }
      }
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full[n & 1]);
    return true;
  };

  if (warp >= kKv4FirstConv) {
    // ------------------------------------------------------------------ convert
    // blocks of unit n, once the scouts know; -1 where they are not to be known
    const auto take_unit = [&](int n) -> int {
      mbar_wait(&unit_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, err, 0x44);
      if (gone()) return -1;
      const int nb = misc[n & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_empty[n & 1]);
      return nb;
    };
    const int ctid = threadIdx.x - 32 * kKv4FirstConv;
    // From two tiles on, half of the warps converts the even tiles and half the odd ones, so that a tile's waits
    // and fences pass beside the other's conversion.  A thread converts, of each of its tiles, the 32 dims
    // [32 part, 32 part + 32) of kItems rows.
    const int part = ctid & 3;
    const int grp_tile = kTi > 1 ? (warp - kKv4FirstConv) / L::kTileWarps : 0;  // its first tile
    const int row0 = (ctid % (32 * L::kTileWarps)) >> 2;
    constexpr int kRowStep = 8 * L::kTileWarps;
    constexpr int kItems = kTcAttnKeys / kRowStep;
    constexpr int kMine = kTi > 1 ? kTi / 2 : 1;  // its tiles: grp_tile + 2 i
    const bool has_part = D >= 128 || part < 2;
    // The codes and group scales of the next block are in flight while its tiles are waited for.
    uint4 raw[kMine][kItems];
    uint32_t grp[kMine][kItems];
    const auto load = [&](uint32_t gb) {
      const uint32_t slot = gb % kKv4Slots;
      mbar_wait(&ent_full[slot], (gb / kKv4Slots) & 1u, abort_flag, err, 0x43);
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int2 ent = ent_s[slot * kTcAttnKeys + row0 + kRowStep * k];
        const uint8_t* base = p.pool.cache + max(ent.x, 0) * page_bytes;
        const uint8_t* codes = base + ent.y * (D / 2) + part * 16 + grp_tile * 64;
        const uint8_t* scales = base + rows * (D / 2) + ent.y * (D / kKv4Group) + part * 2 + grp_tile * 8;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          raw[i][k] = make_uint4(0u, 0u, 0u, 0u);
          grp[i][k] = 0u;
          if (ent.x >= 0 && has_part) {
            raw[i][k] = ld_after_wait(reinterpret_cast<const uint4*>(codes + i * 128));
            grp[i][k] = ld_after_wait(reinterpret_cast<const uint16_t*>(scales + i * 16));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ent_empty[slot]);
    };
    uint32_t gb = 0;  // blocks of this CTA so far
    int n = 0;        // units of this CTA so far
    for (int u = unit0; u < (kSingle ? unit0 + 1 : units); u += unit_step, ++n) {
      int nb = 0;
      if constexpr (kSingle) {  // (the softmax warps, idle so far, bring q)
        nb = take_unit(0);
      } else {
        const int t = u / p.groups;
        const int h0 = (u % p.groups) * kTcAttnHeads;
        bring_q(warp - kKv4FirstConv, n, t, h0, min(kTcAttnHeads, H - h0), [&]() -> bool {
          nb = take_unit(n);
          // q's place is free once the previous unit's score products are done
          if (n > 0 && nb >= 0) mbar_wait(q_empty, static_cast<uint32_t>(n - 1) & 1u, abort_flag, err, 0x41);
          return nb >= 0;
        });
      }
      if (nb < 0) break;
      if (nb > 0) load(gb);
      for (int b = 0; b < nb; ++b, ++gb) {
        if (b % kLook == kLook - 1 && gone()) break;
        const int st = static_cast<int>(gb % kSt);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int m = grp_tile + 2 * i;
          uint8_t* chunk = kv_s + st * L::kStageBytes + (2 * m + (part >> 1)) * L::kChunkBytes;
#pragma unroll
          for (int k = 0; k < kItems; ++k) {
            const int row = row0 + kRowStep * k;
            const uint32_t s2 = e4m3x2_to_f16x2(grp[i][k]);
            const uint32_t w[4] = {raw[i][k].x, raw[i][k].y, raw[i][k].z, raw[i][k].w};
            if (k == 0 && gb >= kSt) mbar_wait(&kv_empty[st * kTi + m], (gb / kSt - 1) & 1u, abort_flag, err, 0x42);
            if (!has_part) continue;
#pragma unroll
            for (int j0 = 0; j0 < 4; ++j0) {
              // the two chunks' threads take their pieces in different order: no bank conflicts
              const int j = (part & 2) ? (j0 ^ 2) : j0;
              const uint32_t s = (j & 2) ? __byte_perm(s2, s2, 0x3232) : __byte_perm(s2, s2, 0x1010);
              uint32_t v[4];
              e2m1x8_to_f16x2((part & 2) ? w[j0 ^ 2] : w[j0], v);
              *reinterpret_cast<uint4*>(chunk + swz128(row, (part & 1) * 64 + j * 16)) =
                  make_uint4(hmul2(v[0], s), hmul2(v[1], s), hmul2(v[2], s), hmul2(v[3], s));
            }
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_full[st * kTi + m]);
        }
        if (b + 1 < nb) load(gb + 1);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax and output
    // The softmax warps meet: in a unit's first block, which all of them enter, at a hardware barrier, later with a limit.
    const auto meet = [&](bool first) {
      if (first) {
        named_bar_sync(kTcEpiBar, kKv4SoftThreads);
        return;
      }
      const uint32_t phase = phase_s[warp - 4];
      __syncwarp();
      if (lane == 0) {
        phase_s[warp - 4] = phase ^ 1u;
        mbar_arrive(soft_all);
      }
      mbar_wait(soft_all, phase, abort_flag, err, 0x68);
    };
    const int etid = threadIdx.x - 128;
    const int quarter = warp & 3;                     // tensor-memory lane quarter
    const int hb = ((warp - 4) >> 2) * kKv4SoftHeads;  // this thread's heads [hb, hb + 16)
    const int r = quarter * 32 + lane;                // key of the block (score rows) / dim of a tile (output rows)
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t gb = 0;
    int n = 0;
    uint32_t checks = 0;  // blocks of this CTA whose bounds were checked
    uint64_t lsum[kKv4SoftHeads / 2];
    if (kSingle && etid < kKv4ConvThreads) {
      const int h0 = (unit0 % p.groups) * kTcAttnHeads;
      bring_q(warp - 4, 0, unit0 / p.groups, h0, min(kTcAttnHeads, H - h0), []() { return true; });
    }
    for (int u = unit0; u < (kSingle ? unit0 + 1 : units); u += unit_step, ++n) {
      const int t = u / p.groups;
      const int h0 = (u % p.groups) * kTcAttnHeads;
      const int nh = min(kTcAttnHeads, H - h0);
      mbar_wait(&unit_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, err, 0x60);
      const int nb = misc[n & 1];
      mbar_wait(&q_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, err, 0x66);  // the q factor
      const float to_log2 = p.scale * 1.4426950408889634f;
      const float* qfac = qfac_s + (n & 1) * kTcAttnHeads;
      constexpr float kQFac = 1.0f / (1 << kKv4QExp);
      if (etid < kTcAttnHeads) max_s[etid] = kKv4NoBound;
#pragma unroll
      for (int h = 0; h < kKv4SoftHeads / 2; ++h) lsum[h] = 0ull;
      if (bar_or(kTcEpiBar, kKv4SoftThreads, *abort_flag != 0)) break;
      if (lane == 0) mbar_arrive(&unit_empty[n & 1]);
      float largest = 0.f;  // row scale of the unit so far
      // the unit's blocks, of q with or without factors of the heads' own (one loop that looks in each block took 3% longer)
      const auto walk = [&](auto with_own) {
        for (int b = 0; b < nb; ++b, ++gb) {
          if (b % kLook == kLook - 1 && gone()) break;
          const uint32_t slot = gb % kKv4Slots;
          mbar_wait(&scl_full[slot], (gb / kKv4Slots) & 1u, abort_flag, err, 0x65);
          float rs = scl_s[slot * kTcAttnKeys + r];
          const float2 span = span_s[slot];
          largest = fmaxf(largest, span.y);
          const bool apart = largest > span.x * kKv4Spread;  // some row's weight may underflow
          __syncwarp();
          if (lane == 0) mbar_arrive(&ent_empty[slot]);
          const bool valid = rs > 0.f;
          float a = to_log2 * (rs * kQFac);                // score to log2 units
          const float lr = valid ? log2f(rs) : -INFINITY;  // a masked key's weight is 0
          const uint64_t lr2 = pack_f32x2(lr, lr);
          const uint32_t s_at = s_tmem + 64 * (gb % kSc) + lane_off + hb;
          mbar_wait(&s_full[gb % kSc], (gb / kSc) & 1u, abort_flag, err, 0x61);
          tc_fence_after_sync();
          float x[kKv4SoftHeads];
          if constexpr (decltype(with_own)::value) {  // the scores with the heads' own q factors, once and for all that follows
            tmem_ld_x16(s_at, x);
            tmem_wait_ld_regs16(x);
#pragma unroll
            for (int h = 0; h < kKv4SoftHeads; ++h) {
              const float f = qfac_s[(n & 1) * kTcAttnHeads + hb + h];
              x[h] *= f > 1.f ? (to_log2 * f) * rs : to_log2 * (f * rs);  // (neither overflows nor vanishes before its time)
            }
            tmem_st_x16(s_at, x);
            tmem_wait_st();
            a = 1.f;
          }
          // exponents relative to the running bounds
          const auto exponents = [&]() {
            const uint64_t minus = pack_f32x2(-1.f, -1.f), a2 = pack_f32x2(a, a);
            tmem_ld_x16(s_at, x);
            tmem_wait_ld_regs16(x);
#pragma unroll
            for (int h = 0; h < kKv4SoftHeads; h += 4) {
              const float4 mv = *reinterpret_cast<const float4*>(max_s + hb + h);
              unpack_f32x2(fma_f32x2(pack_f32x2(mv.x, mv.y), minus, fma_f32x2(pack_f32x2(x[h], x[h + 1]), a2, lr2)), x[h], x[h + 1]);
              unpack_f32x2(fma_f32x2(pack_f32x2(mv.z, mv.w), minus, fma_f32x2(pack_f32x2(x[h + 2], x[h + 3]), a2, lr2)), x[h + 2],
                           x[h + 3]);
            }
          };
          // weights, written into the fp16 row P[key r]; x keeps them
          const auto weights = [&]() {
#pragma unroll
            for (int hh = 0; hh < kKv4SoftHeads; hh += 8) {
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[hh + 2 * i] = exp2_approx(x[hh + 2 * i]);
                x[hh + 2 * i + 1] = exp2_approx(x[hh + 2 * i + 1]);
                const __half2 w = __floats2half2_rn(x[hh + 2 * i], x[hh + 2 * i + 1]);
                pk[i] = *reinterpret_cast<const uint32_t*>(&w);
              }
              *reinterpret_cast<uint4*>(p_s + swz128(r, 2 * (hb + hh))) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          };
          // A unit's first block sets the bounds.  After that the weights are formed with the bounds as they are,
          // while the warps tell one another whether an exponent exceeds its bound by more than 2^8; if one
          // does, which is rare, the bounds are raised and the weights formed again.  (What else is rare goes that way too, as if a
          // bound were exceeded: no branches for all other blocks.)
          bool raise = b == 0;
          if (!raise) {
            exponents();
            float over = x[0];
#pragma unroll
            for (int h = 1; h + 1 < kKv4SoftHeads; h += 2) over = max3(over, x[h], x[h + 1]);
            over = fmaxf(over, x[kKv4SoftHeads - 1]);
            if (__any_sync(0xffffffffu, over > kTcLazyLog2 || apart) && lane == 0) misc[16 + checks % 3] = 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(checked);
            mbar_wait(pv_done, (gb - 1) & 1u, abort_flag, err, 0x63);  // the previous weighted sum has read P
            weights();
            mbar_wait(checked, checks & 1u, abort_flag, err, 0x67);
            raise = __any_sync(0xffffffffu, misc[16 + checks % 3] != 0) != 0;
            ++checks;
            // this flag's next use but one: every warp has read it (two blocks ago), none sets it before the next check
            if (etid == 0) misc[16 + (checks + 1) % 3] = 0;
          }
          if (raise) {
            if (b > 0 && gone()) break;
            const bool far = __any_sync(0xffffffffu, apart) != 0;
            // the largest exponents per head across the 128 keys (the reduction consumes x)
            tmem_ld_x16(s_at, x);
            tmem_wait_ld_regs16(x);
#pragma unroll
            for (int h = 0; h < kKv4SoftHeads; ++h) x[h] = fmaf(x[h], a, lr);
            xpose_reduce16(x, lane, [](float v, float w) { return fmaxf(v, w); });
            if ((lane & 1) == 0) red_s[quarter * kTcAttnHeads + hb + (lane >> 1)] = x[0];
            meet(b == 0);
            if (etid < kTcAttnHeads) {
              const float bm = fmaxf(fmaxf(red_s[etid], red_s[kTcAttnHeads + etid]),
                                     fmaxf(red_s[2 * kTcAttnHeads + etid], red_s[3 * kTcAttnHeads + etid]));
              const float mo = max_s[etid];
              const float mn = (bm > mo + kTcLazyLog2) ? bm : mo;
              // (the root of the factor: a sum may be as large as 2^100 times the bound's unit and is not to be lost)
              alpha_s[etid] = (mo == kKv4NoBound || mn == mo) ? 1.f : exp2f(0.5f * (mo - mn));
              max_s[etid] = mn;
            }
            meet(b == 0);
            if (b > 0) {
              // sums and output accumulators of earlier blocks follow the new bound (this thread: its dim row r
              // of every tile, its 16 head columns)
#pragma unroll
              for (int h = 0; h < kKv4SoftHeads; h += 2) {
                const uint64_t root = pack_f32x2(alpha_s[hb + h], alpha_s[hb + h + 1]);
                lsum[h / 2] = fma_f32x2(fma_f32x2(lsum[h / 2], root, 0ull), root, 0ull);
              }
              tc_fence_after_sync();
#pragma unroll 1
              for (int m = 0; m < kTi; ++m) {
                tmem_ld_x16(o_tmem + lane_off + 64 * m + hb, x);
                tmem_wait_ld_regs16(x);
#pragma unroll
                for (int j = 0; j < kKv4SoftHeads; ++j) x[j] = x[j] * alpha_s[hb + j] * alpha_s[hb + j];
                tmem_st_x16(o_tmem + lane_off + 64 * m + hb, x);
              }
              tmem_wait_st();
            } else if (gb > 0) {
              mbar_wait(pv_done, (gb - 1) & 1u, abort_flag, err, 0x62);
            }
            exponents();
            weights();
            if (far) {  // the denominator's terms by themselves, from the same exponents (the scores are still there)
              exponents();
#pragma unroll
              for (int h = 0; h < kKv4SoftHeads; ++h) x[h] = lr > -INFINITY ? exp2_gradual(x[h] - lr) : 0.f;
              rs = -1.f;
            }
          }
          fence_proxy_async_shared();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full);
          // what makes a weight a term of the denominator (2^-23 off; a division took 1% of a long prompt), or x is the term
          const float inv = rs > 0.f ? rcp_approx(rs) : (rs < 0.f ? 1.f : 0.f);
          const uint64_t inv2 = pack_f32x2(inv, inv);
#pragma unroll
          for (int h = 0; h < kKv4SoftHeads; h += 2) lsum[h / 2] = fma_f32x2(pack_f32x2(x[h], x[h + 1]), inv2, lsum[h / 2]);
        }
      };
      if (__any_sync(0xffffffffu, qfac[lane] != kQFac || qfac[32 + lane] != kQFac))
        walk(std::true_type());
      else
        walk(std::false_type());
      // end of the unit: denominators (partial sums across the 128 keys)
      {
        float l[kKv4SoftHeads];
#pragma unroll
        for (int h = 0; h < kKv4SoftHeads; h += 2) unpack_f32x2(lsum[h / 2], l[h], l[h + 1]);
        xpose_reduce16(l, lane, [](float v, float w) { return v + w; });
        if ((lane & 1) == 0) red_s[quarter * kTcAttnHeads + hb + (lane >> 1)] = l[0];
      }
      named_bar_sync(kTcEpiBar, kKv4SoftThreads);
      if (etid < kTcAttnHeads) {
        const float l = (red_s[etid] + red_s[kTcAttnHeads + etid]) + (red_s[2 * kTcAttnHeads + etid] + red_s[3 * kTcAttnHeads + etid]);
        if (kSingle && shares > 1) {
          float* stats = p.partial_stats + (static_cast<int64_t>(u) * shares + share) * 2 * kTcAttnHeads;
          __stcg(stats + etid, max_s[etid]);
          __stcg(stats + kTcAttnHeads + etid, l);
        } else if (etid < nh) {
          alpha_s[etid] = softmax_factor(max_s[etid], l, p.sink, h0 + etid,
                                         p.lse != nullptr ? p.lse + static_cast<int64_t>(t) * H + h0 + etid : nullptr);
        }
      }
      named_bar_sync(kTcEpiBar, kKv4SoftThreads);
      if (nb > 0) {
        mbar_wait(pv_done, (gb - 1) & 1u, abort_flag, err, 0x64);
        tc_fence_after_sync();
      }
      uint16_t* out = p.out + (static_cast<int64_t>(t) * H + h0) * D;
      const bool row = D >= 128 || quarter < 2;  // (the upper half of a 64-dim row's tile is padding)
      for (int m = 0; m < kTi; ++m) {
        float o[kKv4SoftHeads];
        if (nb > 0 && row) {
          tmem_ld_x16(o_tmem + lane_off + 64 * m + hb, o);
          tmem_wait_ld_regs16(o);
        } else {
#pragma unroll
          for (int j = 0; j < kKv4SoftHeads; ++j) o[j] = 0.f;
        }
        if (kSingle && shares > 1) {
          if (row) {
            float* part = p.partial + (static_cast<int64_t>(u) * shares + share) * kTcAttnHeads * D + 128 * m + r;
#pragma unroll
            for (int j = 0; j < kKv4SoftHeads; ++j) __stcg(part + (hb + j) * D, o[j]);
          }
          continue;
        }
        // Neighbouring lanes (dims) trade halves of a pair of heads, so that each stores two dims of one head: 64
        // contiguous bytes per head and warp, without shared memory or barriers.
        const bool odd = (lane & 1) != 0;
        uint16_t* dst = out + static_cast<int64_t>(hb + (odd ? 1 : 0)) * D + 128 * m + (r & ~1);
#pragma unroll
        for (int j = 0; j < kKv4SoftHeads; j += 2) {
          const float2 f = *reinterpret_cast<const float2*>(alpha_s + hb + j);
          const __nv_bfloat162 two = __floats2bfloat162_rn(o[j] * f.x, o[j + 1] * f.y);
          const uint32_t w = *reinterpret_cast<const uint32_t*>(&two);
          const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 1);
          const uint32_t mine = odd ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
          if (row && hb + j + (odd ? 1 : 0) < nh) *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(j) * D) = mine;
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
      named_bar_sync(kTcEpiBar, kKv4SoftThreads);  // alpha_s and max_s are rewritten by the next unit
    }
  } else if (warp >= 1) {
    // ------------------------------------------------------------------ scout
    uint32_t gb = 0;
    int n = 0;
    for (int u = unit0; u < (kSingle ? unit0 + 1 : units); u += unit_step, ++n) {
      if (gone()) break;
      const int t = u / p.groups;
      const int32_t* list = p.idx + static_cast<int64_t>(t) * p.K;
      const int seq = ld_after_wait(p.seq + t);
      const int start = p.start != nullptr ? ld_after_wait(p.start + t) : 0;
      // blocks to walk: up to the last entry that names a row, looked for from the end
      int last = -1;
      for (int j0 = (p.K - 1) / 256 * 256; j0 >= 0 && last < 0; j0 -= 256) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = j0 + 32 * i + lane < p.K ? ld_after_wait(list + j0 + 32 * i + lane) : -1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (v[i] >= 0) last = j0 + 32 * i + lane;
        last = __reduce_max_sync(0xffffffffu, last);
      }
      if (warp == 2) {  // the unit's q into L2: its loads come when the previous unit's scores are done
        const int nh = min(kTcAttnHeads, H - (u % p.groups) * kTcAttnHeads);
        const uint16_t* q = p.q + (static_cast<int64_t>(t) * H + (u % p.groups) * kTcAttnHeads) * D;
        for (int i = lane; i < nh * (D / 64); i += 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + static_cast<int64_t>(i) * 64));
      }
      const int all = (last + kTcAttnKeys) / kTcAttnKeys;
      const int blk0 = first_block(all, share);
      const int nb = first_block(all, share + 1) - blk0;
      if (warp == 1) {
        if (n > 1) mbar_wait(&unit_empty[n & 1], static_cast<uint32_t>((n >> 1) - 1) & 1u, abort_flag, err, 0x40);
        if (gone()) break;
        if (lane == 0) {
          misc[n & 1] = nb;
          mbar_arrive(&unit_full[n & 1]);
        }
      }
      for (int b = 0; b < nb; ++b, ++gb) {
        if (static_cast<int>(gb % kKv4Scouts) != warp - 1) continue;
        const uint32_t slot = gb % kKv4Slots;
        int2 ent[4];
        float r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = (blk0 + b) * kTcAttnKeys + 32 * i + lane;
          ent[i].x = j < p.K ? ld_after_wait(list + j) : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t pos = static_cast<int64_t>(ent[i].x) - start;
          const bool some = ent[i].x >= 0 && pos >= 0 && pos < INT32_MAX;
          ent[i] = make_int2(some ? kv4_page(p.pool, seq, static_cast<int>(pos)) : -1, static_cast<int>(pos) & (rows - 1));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r[i] = 0.0f;
          if (ent[i].x >= 0)
            r[i] = ld_after_wait(reinterpret_cast<const float*>(p.pool.cache + ent[i].x * page_bytes +
                                                        rows * (D / 2 + D / kKv4Group)) + ent[i].y);
        }
        if (gb >= kKv4Slots) mbar_wait(&ent_empty[slot], (gb / kKv4Slots - 1) & 1u, abort_flag, err, 0x45);
        if (gone()) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) ent_s[slot * kTcAttnKeys + 32 * i + lane] = ent[i];
        mbar_arrive(&ent_full[slot]);
        uint32_t lo = 0x7F7FFFFFu, hi = 0u;  // the block's row scales (as bits: they are positive)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r[i] = ent[i].x >= 0 ? fmaxf(r[i], kKv4MinScale) : 0.0f;
          if (ent[i].x >= 0) lo = min(lo, __float_as_uint(r[i]));
          hi = max(hi, __float_as_uint(r[i]));
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) scl_s[slot * kTcAttnKeys + 32 * i + lane] = r[i];
        if (lane == 0) span_s[slot] = make_float2(__uint_as_float(lo), __uint_as_float(hi));
        mbar_arrive(&scl_full[slot]);
      }
    }
  } else {
    // ------------------------------------------------------------------ MMA issuer (the whole warp, one thread elected)
    const uint32_t on = elect_one();
    const auto wait = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, site)) != 0;
    };
    constexpr uint32_t id_qk = idesc_f16(kTcAttnKeys, kTcAttnHeads, false, false);
    constexpr uint32_t id_pv = idesc_f16(128, kTcAttnHeads, true, true);
    const uint64_t kv_k = desc_sw128(smem_addr(kv_s), 16, 1024);               // K-major: keys x dims
    const uint64_t q_k = desc_sw128(smem_addr(q_s), 16, 1024);                 // K-major: heads x dims
    const uint64_t kv_mn = desc_sw128(smem_addr(kv_s), L::kChunkBytes, 1024);  // MN-major: dims x keys
    const uint64_t p_mn = desc_sw128(smem_addr(p_s), 16384, 1024);             // MN-major: heads x keys
    // S^T of block gb over D / 16 steps; chunk c holds dims [64 c, 64 c + 64)
    const auto score = [&](uint32_t gb) -> bool {
      const uint32_t st = gb % kSt;
      const uint64_t a = kv_k + st * (L::kStageBytes >> 4);
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        if ((c & 1) == 0) {
          if (!wait(&kv_full[st * kTi + c / 2], (gb / kSt) & 1u, 0x53)) return false;
          tc_fence_after_sync();
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t ad = a + ((c * L::kChunkBytes + kk * 32) >> 4), bd = q_k + ((c * L::kQChunkBytes + kk * 32) >> 4);
          if (c == 0 && kk == 0)
            mma_f16_if<false>(on, s_tmem + 64 * (gb % kSc), ad, bd, id_qk, 0u);
          else
            mma_f16_if<true>(on, s_tmem + 64 * (gb % kSc), ad, bd, id_qk);
        }
      }
      mma_commit_if(on, &s_full[gb % kSc]);
      return true;
    };
    uint32_t gb = 0;
    int n = 0;
    bool ok = true;
    for (int u = unit0; ok && u < (kSingle ? unit0 + 1 : units); u += unit_step, ++n) {
      if (!wait(&unit_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, 0x50)) break;
      const int nb = __shfl_sync(0xffffffffu, misc[n & 1], 0);
      if (lane == 0) mbar_arrive(&unit_empty[n & 1]);
      __syncwarp();
      if (!wait(&q_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, 0x51)) break;
      if (nb > 0 && !score(gb)) break;
      if (nb <= 1) mma_commit_if(on, q_empty);  // (after the unit's last score product)
      for (int b = 0; b < nb; ++b, ++gb) {
        if (kSt > 1 && b + 1 < nb) {
          if (!score(gb + 1)) {
            ok = false;
            break;
          }
          if (b + 2 == nb) mma_commit_if(on, q_empty);
        }
        if (!wait(p_full, gb & 1u, 0x54)) {
          ok = false;
          break;
        }
        // the unit's first weighted sum overwrites O: the previous unit's output must be read
        if (b == 0 && n > 0 && !wait(o_empty, static_cast<uint32_t>(n - 1) & 1u, 0x52)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t st = gb % kSt;
        const uint64_t a = kv_mn + st * (L::kStageBytes >> 4);
        const uint32_t more = b > 0 ? 1u : 0u;
#pragma unroll
        for (int m = 0; m < kTi; ++m) {
#pragma unroll
          for (int ks = 0; ks < kTcAttnKeys / 16; ++ks) {
            const uint64_t ad = a + ((2 * m * L::kChunkBytes + ks * 16 * 128) >> 4), bd = p_mn + ((ks * 16 * 128) >> 4);
            if (ks == 0)
              mma_f16_if<false>(on, o_tmem + 64 * m, ad, bd, id_pv, more);
            else
              mma_f16_if<true>(on, o_tmem + 64 * m, ad, bd, id_pv);
          }
          mma_commit_if(on, &kv_empty[st * kTi + m]);
        }
        mma_commit_if(on, pv_done);
        if (kSt == 1 && b + 1 < nb) {
          if (!score(gb + 1)) {
            ok = false;
            break;
          }
          if (b + 2 == nb) mma_commit_if(on, q_empty);
        }
      }
    }
    // every MMA issued by this thread has completed once `drain` flips
    mma_commit_if(on, drain);
    mbar_wait_drain(drain, 0);
    __syncwarp();
  }

  if (kSingle && shares > 1) {
    // ------------------------------------------------------------------ join
    __syncthreads();
    cluster_sync_all();
    const int t = unit0 / p.groups;
    const int h0 = (unit0 % p.groups) * kTcAttnHeads;
    const int nh = min(kTcAttnHeads, H - h0);
    // This CTA's share of the group's [64][D] outputs, four dims at a time.  Partial outputs, bounds and sums pass
    // through L2: read from the other CTAs' shared memory instead, 128 KB arrive at 13 bytes a clock (10,000 cycles at
    // D = 512).  The first loads are in flight while the shares' factors are formed.
    constexpr int kAll = kTcAttnHeads * D / 4;
    constexpr int kPart = 8;  // partial outputs in flight per thread
    const int per = (kAll + shares - 1) / shares;
    const int end = min(min(kAll, (share + 1) * per), nh * (D / 4));
    const float4* part = reinterpret_cast<const float4*>(p.partial) + static_cast<int64_t>(unit0) * shares * kAll;
    const float* stats = p.partial_stats + static_cast<int64_t>(unit0) * shares * 2 * kTcAttnHeads;
    uint16_t* out = p.out + (static_cast<int64_t>(t) * H + h0) * D;
    int i = share * per + threadIdx.x;
    float4 v[kPart];
    const auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < kPart; ++k) {
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < end && k0 + k < shares) v[k] = __ldcg(part + static_cast<int64_t>(k0 + k) * kAll + i);
      }
    };
    fetch(0);
    float* sum_s = reinterpret_cast<float*>(p_s);  // [shares][64] sums (P's place: every product is done)
    for (int j = threadIdx.x; j < shares * kTcAttnHeads; j += kKv4Threads) {
      const float* at = stats + (j / kTcAttnHeads) * 2 * kTcAttnHeads + j % kTcAttnHeads;
      join_s[j] = __ldcg(at);
      sum_s[j] = __ldcg(at + kTcAttnHeads);
    }
    __syncthreads();
    if (threadIdx.x < nh) {
      const int h = threadIdx.x;
      float top = kKv4NoBound, sum = 0.f;
#pragma unroll 4
      for (int k = 0; k < shares; ++k) top = fmaxf(top, join_s[k * kTcAttnHeads + h]);
#pragma unroll 4
      for (int k = 0; k < shares; ++k) {
        const float m = join_s[k * kTcAttnHeads + h];
        const float root = m == kKv4NoBound ? 0.f : exp2f(0.5f * (m - top));  // (as where a bound is raised)
        sum = fmaf(sum_s[k * kTcAttnHeads + h] * root, root, sum);
        join_s[k * kTcAttnHeads + h] = root * root;
      }
      alpha_s[h] = softmax_factor(top, sum, p.sink, h0 + h,
                                  p.lse != nullptr && share == 0 ? p.lse + static_cast<int64_t>(t) * H + h0 + h : nullptr);
    }
    __syncthreads();
    for (; i < end; i += kKv4Threads) {
      const int h = i / (D / 4);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k0 = 0; k0 < shares; k0 += kPart) {
        if (k0 > 0 || i >= share * per + kKv4Threads) fetch(k0);
#pragma unroll
        for (int k = 0; k < kPart; ++k) {
          const float w = k0 + k < shares ? join_s[(k0 + k) * kTcAttnHeads + h] : 0.f;
          acc.x = fmaf(v[k].x, w, acc.x);
          acc.y = fmaf(v[k].y, w, acc.y);
          acc.z = fmaf(v[k].z, w, acc.z);
          acc.w = fmaf(v[k].w, w, acc.w);
        }
      }
      const float f = alpha_s[h];
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * f, acc.y * f), hi = __floats2bfloat162_rn(acc.z * f, acc.w * f);
      *reinterpret_cast<uint2*>(out + static_cast<int64_t>(i) * 4) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tbase, L::kTmemCols);
}

}  // namespace dsa
