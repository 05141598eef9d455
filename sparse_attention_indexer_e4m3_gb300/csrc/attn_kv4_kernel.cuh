// Sparse attention over the 4-bit paged cache on the tensor cores.  For query token t and head h, over
// the entries of idx[t, :] that name a mapped row j of the token's sequence (kv_j = r_j * v_j, v_j the
// exact fp16 values s * c of kv4.cuh):
//     x_j = scale * q[t,h,:] . kv_j
//     out[t,h,:] = sum_j e^{x_j} kv_j / ( sum_j e^{x_j} + e^{sink[h]} )
// Both products run on fp16 operands with fp32 accumulators.  v_j is exact; q is bf16 and becomes fp16
// exactly (times a power of two of the token where its largest value is not in [1, 2^15), values more than
// 2^29 below the largest rounded); the weights enter the second product as w_j = r_j * 2^(y_j - m), y = x log2 e,
// rounded to fp16 (half a step, 2^-11), with m a bound on y_j + log2 r_j so that w_j <= 2^8 whatever the
// row scales are.  The denominator sums w_j / r_j in fp32.  fp16 weights rather than bf16 ones because
// their rounding would otherwise be as large as the output's own.
//
// A unit is (token, group of up to 64 heads, share of the token's list); a cluster of S CTAs shares
// one list and joins its S partial results through distributed shared memory, so a call with few tokens still
// uses most SMs and needs no second launch.  One CTA per SM, 512 threads, per block of 128 entries:
//   gather   (warps 12-15) looks the entries' pages up, converts the rows' codes to fp16 values and
//                          writes them as D / 64 chunks of [128 keys x 128 bytes], 128-byte swizzled; a
//                          masked entry becomes a row of zeros (its memory is not read);
//   score    (warp 0)      S^T = V . Q^T: M = 128 keys, N = 64 heads, K = D (tcgen05.mma kind::f16);
//   softmax  (warps 4-11)  thread = (key, 32 heads): weights as fp16 rows P[key][head]; the running
//                          bound m moves only when exceeded by more than 2^8;
//   weighted (warp 0)      O^T += V^T . P^T: M = 128 output dims (D / 128 tiles), N = 64, K = 128 keys.
// The gather refills a tile of 128 dims as soon as the weighted sum has read it; its global loads for the
// next block are in flight while it waits.
#pragma once

#include <cuda_fp16.h>

#include "attn_tc_kernel.cuh"
#include "cluster.cuh"
#include "kv4.cuh"

namespace dsa {

// Row scales outside this range are clamped (the quantiser writes 2^-100 to 2^117).
constexpr float kKv4MinScale = 7.888609052210118e-31f;  // 2^-100

template <int D>
struct AttnKv4Layout {
  static constexpr int kChunks = D / 64;                        // chunks of a row in the score product
  static constexpr int kTiles = D >= 128 ? D / 128 : 1;         // output tiles (D = 64: half of one is zero)
  static constexpr int kChunkBytes = kTcAttnKeys * 128;
  static constexpr int kQChunkBytes = kTcAttnHeads * 128;
  static constexpr int kKv = 0;
  static constexpr int kQ = kKv + 2 * kTiles * kChunkBytes;
  static constexpr int kP = kQ + kChunks * kQChunkBytes;        // fp16 [128 keys][64 heads]
  static constexpr int kEnt = kP + kTcAttnKeys * 128;           // int2 [2][128]: page, row in the page
  static constexpr int kScl = kEnt + 2 * kTcAttnKeys * 8;       // float [2][128]: row scale, 0 = masked
  static constexpr int kRed = kScl + 2 * kTcAttnKeys * 4;       // float [4][64] cross-warp scratch
  static constexpr int kMax = kRed + 4 * kTcAttnHeads * 4;      // float [64] running bound (log2 units)
  static constexpr int kAlpha = kMax + kTcAttnHeads * 4;        // float [64] rescale / output factors
  static constexpr int kSum = kAlpha + kTcAttnHeads * 4;        // float [64] denominators (of this share)
  static constexpr int kJoin = kSum + kTcAttnHeads * 4;         // float [8][64] factors of the shares
  static constexpr int kMisc = kJoin + 8 * kTcAttnHeads * 4;    // int [32]
  static constexpr int kBar = kMisc + 128;
  static constexpr int kNumBars = 10 + 2 * kTiles;
  static constexpr int kSmem = kBar + kNumBars * 8 + 1024;      // + alignment slack
  // the joined shares' partial outputs, fp32 [D][64], take the place of the kv block
  static_assert(D * kTcAttnHeads * 4 <= 2 * kTiles * kChunkBytes, "partial outputs fit the kv block");
  static constexpr int kTmemCols = kTiles == 1 ? 128 : (kTiles == 2 ? 256 : 512);
};

// Instruction descriptor, kind::f16 with fp16 operands and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Index of the 16-byte piece of dim d's row that holds heads [4 u, 4 u + 4) of the partial outputs: the
// pieces of neighbouring dims fall on different banks.
__device__ __forceinline__ uint32_t join_at(int d, int u) { return static_cast<uint32_t>(d * 16 + (u ^ (d & 15))); }

// Output factor of a head whose weights' bound is m (log2 units) and whose denominator, in units of
// 2^m, is l without the sink; writes the natural log of the whole denominator where lse is given.  0 for
// a head without keys and sink.  The larger of bound and sink is the unit, so neither overflows.
__device__ __forceinline__ float softmax_factor(float m, float l, const float* sink, int h, float* lse) {
  const bool keys = m != -INFINITY;
  float f = keys ? 1.f : 0.f, unit = m;
  if (!keys) l = 0.f;
  if (sink != nullptr) {
    const float s2 = __ldg(sink + h) * 1.4426950408889634f;
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

// Two bf16 values to fp16, times f.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float f) {
  const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D>
__global__ void __launch_bounds__(kTcAttnThreads, 1) sparse_attn_kv4_kernel(const AttnKv4Params p, int shares,
                                                                            unsigned* err) {
  using L = AttnKv4Layout<D>;
  constexpr int kCh = L::kChunks;
  constexpr int kTi = L::kTiles;
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
  float* sum_s = reinterpret_cast<float*>(smem + L::kSum);
  float* join_s = reinterpret_cast<float*>(smem + L::kJoin);
  // [0] blocks of the unit in flight, [1] the bits of its q factor, [2] / [3] their copies for the softmax
  // warps, [4] / [5] for the gather warps, [8..15] the gather warps' partial results
  volatile int* misc = reinterpret_cast<volatile int*>(smem + L::kMisc);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* s_full = bars + 2;
  uint64_t* p_full = bars + 3;
  uint64_t* pv_done = bars + 4;
  uint64_t* o_empty = bars + 5;
  uint64_t* tok_full = bars + 6;  // one unit in flight between the gather and the rest
  uint64_t* tok_empty = bars + 7;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* kv_full = bars + 9;
  uint64_t* kv_empty = kv_full + kTi;
  uint64_t* drain = kv_empty + kTi;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int H = p.H;
  const int units = p.T * p.groups;
  const int share = static_cast<int>(blockIdx.x) % shares;
  const int unit0 = static_cast<int>(blockIdx.x) / shares;
  const int unit_step = static_cast<int>(gridDim.x) / shares;

  // q rows past the group's heads, and the upper half of a 64-dim row's tile, stay zero
  for (int i = threadIdx.x; i < kCh * L::kQChunkBytes / 16; i += kTcAttnThreads)
    reinterpret_cast<uint4*>(q_s)[i] = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (D == 64) {
    for (int i = threadIdx.x; i < L::kChunkBytes / 16; i += kTcAttnThreads)
      reinterpret_cast<uint4*>(kv_s + L::kChunkBytes)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (threadIdx.x == 0) {
    mbar_init(q_full, kTcGatherThreads);
    mbar_init(q_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, kTcSoftThreads);
    mbar_init(pv_done, 1);
    mbar_init(o_empty, kTcSoftThreads);
    mbar_init(tok_full, 1);
    mbar_init(tok_empty, 2);  // the MMA issuer and the softmax warps
    for (int m = 0; m < kTi; ++m) {
      mbar_init(&kv_full[m], kTcGatherThreads);
      mbar_init(&kv_empty[m], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  fence_proxy_async_shared();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const uint32_t s_tmem = tbase;
  const uint32_t o_tmem = tbase + 64;

  if (warp >= 12) {
    // ------------------------------------------------------------------ gather
    const int gtid = threadIdx.x - 384;
    const int rows = 1 << p.pool.log_rows;
    const int64_t page_bytes = static_cast<int64_t>(rows) * kv4_row_bytes(D);
    // Thread gtid converts, of every tile, the 32 dims [32 part, 32 part + 32) of rows gtid / 4 + 32 k.
    const int part = gtid & 3;
    const int row0 = gtid >> 2;
    const bool has_part = D >= 128 || part < 2;
    uint32_t gb = 0;  // blocks of this CTA so far
    int n = 0;        // units of this CTA so far
    for (int u = unit0; u < units; u += unit_step, ++n) {
      const int t = u / p.groups;
      const int h0 = (u % p.groups) * kTcAttnHeads;
      const int nh = min(kTcAttnHeads, H - h0);
      const int32_t* list = p.idx + static_cast<int64_t>(t) * p.K;
      const int seq = __ldg(p.seq + t);
      const int start = p.start != nullptr ? __ldg(p.start + t) : 0;
      // blocks to walk: up to the last entry that names a row
      int last = -1;
      for (int j = gtid; j < p.K; j += kTcGatherThreads)
        if (__ldg(list + j) >= 0) last = j;
      last = __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) misc[8 + (warp - 12)] = last;
      named_bar_sync(kTcGatherBar, kTcGatherThreads);
      const int nball = (max(max(misc[8], misc[9]), max(misc[10], misc[11])) + kTcAttnKeys) / kTcAttnKeys;
      const int blk0 = static_cast<int>(static_cast<int64_t>(nball) * share / shares);
      const int nb = static_cast<int>(static_cast<int64_t>(nball) * (share + 1) / shares) - blk0;
      // the unit's q as fp16 once the previous unit's score products are done
      if (n > 0) mbar_wait(q_empty, static_cast<uint32_t>(n - 1) & 1u, abort_flag, err, 0x41);
      float f = 1.0f;
      for (int pass = 0; pass < 2; ++pass) {
        uint32_t top = 0u;
        const uint16_t* q = p.q + (static_cast<int64_t>(t) * H + h0) * D;
#pragma unroll 4
        for (int i = gtid; i < kTcAttnHeads * (D / 8); i += kTcGatherThreads) {
          const int h = i / (D / 8), pc = i % (D / 8);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (h < nh) v = __ldg(reinterpret_cast<const uint4*>(q + static_cast<int64_t>(h) * D) + pc);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
          *reinterpret_cast<uint4*>(q_s + (pc / 8) * L::kQChunkBytes + swz128(h, (pc % 8) * 16)) =
              make_uint4(bf16x2_to_f16x2(v.x, f), bf16x2_to_f16x2(v.y, f), bf16x2_to_f16x2(v.z, f), bf16x2_to_f16x2(v.w, f));
        }
        if (pass == 1) break;
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) misc[12 + (warp - 12)] = static_cast<int>(top);
        named_bar_sync(kTcGatherBar, kTcGatherThreads);
        const int e = (max(max(misc[12], misc[13]), max(misc[14], misc[15])) >> 7) - 127;  // exponent of the largest
        if (e >= 0 && e < 15) break;
        if (e < -126 || e > 127) break;  // zeros (or less than the least normal number), or not finite
        f = __int_as_float((127 + min(13 - e, 126)) << 23);  // the largest lands in [2^13, 2^14)
      }
      if (gtid == 0) {
        mbar_wait(tok_empty, (static_cast<uint32_t>(n) & 1u) ^ 1u, abort_flag, err, 0x40);
        misc[0] = nb;
        misc[1] = __float_as_int(f);
        mbar_arrive(tok_full);
      }
      fence_proxy_async_shared();
      mbar_arrive(q_full);

      // entry of key gtid of block b, and its row scale
      const auto lookup = [&](int b, int2& ent, float& r) {
        const int j = (blk0 + b) * kTcAttnKeys + gtid;
        const int v = b < nb && j < p.K ? __ldg(list + j) : -1;
        const int64_t pos = static_cast<int64_t>(v) - start;
        const int page = v >= 0 && pos >= 0 && pos < INT32_MAX ? kv4_page(p.pool, seq, static_cast<int>(pos)) : -1;
        ent = make_int2(page, static_cast<int>(pos) & (rows - 1));
        r = 0.0f;
        if (page >= 0)
          r = __ldg(reinterpret_cast<const float*>(p.pool.cache + page * page_bytes + rows * (D / 2 + D / kKv4Group)) + ent.y);
      };
      uint4 raw[kTi][4];
      uint32_t grp[kTi][4];
      const auto load = [&](uint32_t slot) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int2 ent = ent_s[(slot & 1u) * kTcAttnKeys + row0 + 32 * k];
          const uint8_t* base = p.pool.cache + max(ent.x, 0) * page_bytes;
          const uint8_t* codes = base + ent.y * (D / 2) + part * 16;
          const uint8_t* scales = base + rows * (D / 2) + ent.y * (D / kKv4Group) + part * 2;
#pragma unroll
          for (int m = 0; m < kTi; ++m) {
            raw[m][k] = make_uint4(0u, 0u, 0u, 0u);
            grp[m][k] = 0u;
            if (ent.x >= 0 && has_part) {
              raw[m][k] = __ldg(reinterpret_cast<const uint4*>(codes + m * 64));
              grp[m][k] = __ldg(reinterpret_cast<const uint16_t*>(scales + m * 8));
            }
          }
        }
      };
      int2 ent;
      float r;
      lookup(0, ent, r);
      if (nb > 0) {
        ent_s[(gb & 1u) * kTcAttnKeys + gtid] = ent;
        scl_s[(gb & 1u) * kTcAttnKeys + gtid] = ent.x >= 0 ? fmaxf(r, kKv4MinScale) : 0.0f;
        named_bar_sync(kTcGatherBar, kTcGatherThreads);
        load(gb);
      }
      for (int b = 0; b < nb; ++b, ++gb) {
        lookup(b + 1, ent, r);
#pragma unroll
        for (int m = 0; m < kTi; ++m) {
          if (gb > 0) mbar_wait(&kv_empty[m], (gb - 1) & 1u, abort_flag, err, 0x42);
          if (has_part) {
            uint8_t* chunk = kv_s + (2 * m + (part >> 1)) * L::kChunkBytes;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = row0 + 32 * k;
              const uint32_t s2 = e4m3x2_to_f16x2(grp[m][k]);
              const uint32_t w[4] = {raw[m][k].x, raw[m][k].y, raw[m][k].z, raw[m][k].w};
#pragma unroll
              for (int i0 = 0; i0 < 4; ++i0) {
                // the two chunks' threads take their pieces in different order: no bank conflicts
                const int i = (part & 2) ? (i0 ^ 2) : i0;
                const uint32_t wi = (part & 2) ? w[i0 ^ 2] : w[i0];
                const uint32_t s = (i & 2) ? __byte_perm(s2, s2, 0x3232) : __byte_perm(s2, s2, 0x1010);
                uint32_t v[4];
                e2m1x8_to_f16x2(wi, v);
                *reinterpret_cast<uint4*>(chunk + swz128(row, (part & 1) * 64 + i * 16)) =
                    make_uint4(hmul2(v[0], s), hmul2(v[1], s), hmul2(v[2], s), hmul2(v[3], s));
              }
            }
          }
          fence_proxy_async_shared();
          mbar_arrive(&kv_full[m]);
        }
        // the next block's entries: the softmax of block gb - 1, whose slot this is, is finished, since
        // the weighted sum of that block, awaited above, followed it
        if (b + 1 < nb) {
          ent_s[((gb + 1) & 1u) * kTcAttnKeys + gtid] = ent;
          scl_s[((gb + 1) & 1u) * kTcAttnKeys + gtid] = ent.x >= 0 ? fmaxf(r, kKv4MinScale) : 0.0f;
          named_bar_sync(kTcGatherBar, kTcGatherThreads);
          load(gb + 1);
        }
      }
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t id_qk = idesc_f16(kTcAttnKeys, kTcAttnHeads, false, false);
      const uint32_t id_pv = idesc_f16(128, kTcAttnHeads, true, true);
      const uint64_t kv_k = desc_sw128(smem_addr(kv_s), 16, 1024);               // K-major: keys x dims
      const uint64_t q_k = desc_sw128(smem_addr(q_s), 16, 1024);                 // K-major: heads x dims
      const uint64_t kv_mn = desc_sw128(smem_addr(kv_s), L::kChunkBytes, 1024);  // MN-major: dims x keys
      const uint64_t p_mn = desc_sw128(smem_addr(p_s), 16384, 1024);             // MN-major: heads x keys
      uint32_t gb = 0;
      int n = 0;
      bool ok = true;
      for (int u = unit0; ok && u < units; u += unit_step, ++n) {
        if (!mbar_wait(tok_full, static_cast<uint32_t>(n) & 1u, abort_flag, err, 0x50)) break;
        const int nb = misc[0];
        mbar_arrive(tok_empty);
        if (!mbar_wait(q_full, static_cast<uint32_t>(n) & 1u, abort_flag, err, 0x51)) break;
        for (int b = 0; b < nb; ++b, ++gb) {
          for (int c = 0; c < kCh; ++c) {
            if ((c & 1) == 0) {
              if (!mbar_wait(&kv_full[c / 2], gb & 1u, abort_flag, err, 0x53)) {
                ok = false;
                break;
              }
              tc_fence_after_sync();
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(s_tmem, kv_k + ((c * L::kChunkBytes + kk * 32) >> 4), q_k + ((c * L::kQChunkBytes + kk * 32) >> 4),
                       id_qk, (c | kk) ? 1u : 0u);
          }
          if (!ok) break;
          mma_commit(s_full);
          if (!mbar_wait(p_full, gb & 1u, abort_flag, err, 0x54)) {
            ok = false;
            break;
          }
          // the unit's first weighted sum overwrites O: the previous unit's output must be read
          if (b == 0 && n > 0 && !mbar_wait(o_empty, static_cast<uint32_t>(n - 1) & 1u, abort_flag, err, 0x52)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          for (int m = 0; m < kTi; ++m) {
#pragma unroll
            for (int ks = 0; ks < kTcAttnKeys / 16; ++ks)
              mma_bf16(o_tmem + 64 * m, kv_mn + ((2 * m * L::kChunkBytes + ks * 16 * 128) >> 4),
                       p_mn + ((ks * 16 * 128) >> 4), id_pv, (b > 0 || ks > 0) ? 1u : 0u);
            mma_commit(&kv_empty[m]);
          }
          mma_commit(pv_done);
        }
        if (!ok) break;
        mma_commit(q_empty);
      }
      // every MMA issued by this thread has completed once `drain` flips
      mma_commit(drain);
      mbar_wait_drain(drain, 0);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax and output
    const int etid = threadIdx.x - 128;
    const int quarter = warp & 3;                     // tensor-memory lane quarter
    const int hb = ((warp - 4) >> 2) * kTcHalfHeads;  // this thread's heads [hb, hb + 32)
    const int r = quarter * 32 + lane;                // key of the block (score rows) / dim of a tile (output rows)
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t gb = 0;
    int n = 0;
    float lsum[kTcHalfHeads];
    for (int u = unit0; u < units; u += unit_step, ++n) {
      const int t = u / p.groups;
      const int h0 = (u % p.groups) * kTcAttnHeads;
      const int nh = min(kTcAttnHeads, H - h0);
      if (etid == 0) {
        mbar_wait(tok_full, static_cast<uint32_t>(n) & 1u, abort_flag, err, 0x60);
        misc[2] = misc[0];
        misc[3] = misc[1];
        mbar_arrive(tok_empty);
      }
      if (etid < kTcAttnHeads) max_s[etid] = -INFINITY;
#pragma unroll
      for (int h = 0; h < kTcHalfHeads; ++h) lsum[h] = 0.f;
      named_bar_sync(kTcEpiBar, kTcSoftThreads);
      const int nb = misc[2];
      const float to_log2 = p.scale * 1.4426950408889634f / __int_as_float(misc[3]);
      for (int b = 0; b < nb; ++b, ++gb) {
        mbar_wait(&kv_full[0], gb & 1u, abort_flag, err, 0x65);  // the block's row scales
        const float rs = scl_s[(gb & 1u) * kTcAttnKeys + r];
        const bool valid = rs > 0.f;
        const float a = to_log2 * rs;                       // score to log2 units
        const float lr = valid ? log2f(rs) : -INFINITY;     // a masked key's weight is 0
        const float inv = valid ? 1.0f / rs : 0.f;
        mbar_wait(s_full, gb & 1u, abort_flag, err, 0x61);
        tc_fence_after_sync();
        float x[kTcHalfHeads];
        tmem_ld_x32_sync(s_tmem + lane_off + hb, x);
#pragma unroll
        for (int h = 0; h < kTcHalfHeads; ++h) x[h] = fmaf(x[h], a, lr);
        // does a value exceed its head's running bound by more than 2^8 (or is it the first)?
        bool exceed = false;
#pragma unroll
        for (int h = 0; h < kTcHalfHeads; h += 4) {
          const float4 mv = *reinterpret_cast<const float4*>(max_s + hb + h);
          exceed |= (x[h] > mv.x + kTcLazyLog2) | (x[h + 1] > mv.y + kTcLazyLog2) | (x[h + 2] > mv.z + kTcLazyLog2) |
                    (x[h + 3] > mv.w + kTcLazyLog2);
        }
        const bool raise = bar_or(kTcEpiBar, kTcSoftThreads, exceed);
        if (raise) {
          // (the reduction consumes x; the scores are read again from tensor memory below)
          xpose_reduce32(x, lane, [](float a2, float c) { return fmaxf(a2, c); });
          red_s[quarter * kTcAttnHeads + hb + lane] = x[0];
          named_bar_sync(kTcEpiBar, kTcSoftThreads);
          if (etid < kTcAttnHeads) {
            const float bm = fmaxf(fmaxf(red_s[etid], red_s[kTcAttnHeads + etid]),
                                   fmaxf(red_s[2 * kTcAttnHeads + etid], red_s[3 * kTcAttnHeads + etid]));
            const float mo = max_s[etid];
            const float mn = (bm > mo + kTcLazyLog2) ? bm : mo;
            alpha_s[etid] = (mo == -INFINITY || mn == mo) ? 1.f : exp2f(mo - mn);
            max_s[etid] = mn;
          }
          named_bar_sync(kTcEpiBar, kTcSoftThreads);
          bool rescale = false;
#pragma unroll
          for (int h = 0; h < kTcHalfHeads; ++h) {
            const float al = alpha_s[hb + h];
            lsum[h] *= al;
            rescale |= al != 1.f;
          }
          // the output accumulators of earlier blocks follow the new bound (this thread: its dim row r
          // of every tile, its 32 head columns)
          rescale = bar_or(kTcEpiBar, kTcSoftThreads, rescale);
          if (b > 0 && rescale) {
            mbar_wait(pv_done, (gb - 1) & 1u, abort_flag, err, 0x62);
            tc_fence_after_sync();
            for (int m = 0; m < kTi; ++m) {
#pragma unroll
              for (int c = 0; c < kTcHalfHeads; c += 16) {
                float o[16];
                tmem_ld_x16(o_tmem + lane_off + 64 * m + hb + c, o);
                tmem_wait_ld_regs16(o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= alpha_s[hb + c + j];
                tmem_st_x16(o_tmem + lane_off + 64 * m + hb + c, o);
              }
            }
            tmem_wait_st();
          }
          tmem_ld_x32_sync(s_tmem + lane_off + hb, x);
#pragma unroll
          for (int h = 0; h < kTcHalfHeads; ++h) x[h] = fmaf(x[h], a, lr);
        }
        // weights, written into the fp16 row P[key r] once the previous block's weighted sum has read P
        if (gb > 0) mbar_wait(pv_done, (gb - 1) & 1u, abort_flag, err, 0x63);
#pragma unroll
        for (int hh = 0; hh < kTcHalfHeads; hh += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            const float4 mv = *reinterpret_cast<const float4*>(max_s + hb + hh + 4 * q2);
            const float mu[4] = {mv.x, mv.y, mv.z, mv.w};
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int h = hh + 4 * q2 + i;
              e[i] = exp2_approx(x[h] - (mu[i] == -INFINITY ? 0.f : mu[i]));
              lsum[h] = fmaf(e[i], inv, lsum[h]);
            }
            const __half2 lo = __floats2half2_rn(e[0], e[1]);
            const __half2 hi = __floats2half2_rn(e[2], e[3]);
            pk[2 * q2] = *reinterpret_cast<const uint32_t*>(&lo);
            pk[2 * q2 + 1] = *reinterpret_cast<const uint32_t*>(&hi);
          }
          *reinterpret_cast<uint4*>(p_s + swz128(r, 2 * (hb + hh))) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        fence_proxy_async_shared();
        tc_fence_before_sync();
        mbar_arrive(p_full);
      }
      // end of the unit: denominators (partial sums across the 128 keys)
      xpose_reduce32(lsum, lane, [](float a2, float c) { return a2 + c; });
      red_s[quarter * kTcAttnHeads + hb + lane] = lsum[0];
      named_bar_sync(kTcEpiBar, kTcSoftThreads);
      if (etid < kTcAttnHeads) {
        const float l = (red_s[etid] + red_s[kTcAttnHeads + etid]) + (red_s[2 * kTcAttnHeads + etid] + red_s[3 * kTcAttnHeads + etid]);
        if (shares > 1) {
          sum_s[etid] = l;
        } else if (etid < nh) {
          alpha_s[etid] = softmax_factor(max_s[etid], l, p.sink, h0 + etid,
                                         p.lse != nullptr ? p.lse + static_cast<int64_t>(t) * H + h0 + etid : nullptr);
        }
      }
      named_bar_sync(kTcEpiBar, kTcSoftThreads);
      if (nb > 0) {
        mbar_wait(pv_done, (gb - 1) & 1u, abort_flag, err, 0x64);
        tc_fence_after_sync();
      }
      uint16_t* out = p.out + (static_cast<int64_t>(t) * H + h0) * D;
      for (int m = 0; m < kTi; ++m) {
        const int d = 128 * m + r;
        if (D == 64 && quarter >= 2) break;  // (warp-uniform: the tile's upper half is padding)
#pragma unroll
        for (int c = 0; c < kTcHalfHeads; c += 16) {
          float o[16];
          if (nb > 0) {
            tmem_ld_x16(o_tmem + lane_off + 64 * m + hb + c, o);
            tmem_wait_ld_regs16(o);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = 0.f;
          }
          if (shares > 1) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              reinterpret_cast<float4*>(kv_s)[join_at(d, (hb + c + j) / 4)] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int h = hb + c + j;
              if (h < nh) {
                const __nv_bfloat16 ob = __float2bfloat16_rn(o[j] * alpha_s[h]);
                out[static_cast<int64_t>(h) * D + d] = *reinterpret_cast<const uint16_t*>(&ob);
              }
            }
          }
        }
      }
      tc_fence_before_sync();
      mbar_arrive(o_empty);
      named_bar_sync(kTcEpiBar, kTcSoftThreads);  // alpha_s, max_s and misc are rewritten by the next unit
    }
  }

  if (shares > 1) {
    // ------------------------------------------------------------------ join (one unit per cluster)
    __syncthreads();
    cluster_sync_all();
    const int t = unit0 / p.groups;
    const int h0 = (unit0 % p.groups) * kTcAttnHeads;
    const int nh = min(kTcAttnHeads, H - h0);
    if (threadIdx.x < kTcAttnHeads) {
      const int h = threadIdx.x;
      float m[8], l[8];
      float top = -INFINITY;
      for (int i = 0; i < shares; ++i) {
        m[i] = ld_cluster_f32(smem_addr(max_s + h), i);
        l[i] = ld_cluster_f32(smem_addr(sum_s + h), i);
        top = fmaxf(top, m[i]);
      }
      float sum = 0.f;
      for (int i = 0; i < shares; ++i) {
        m[i] = m[i] == -INFINITY ? 0.f : exp2f(m[i] - top);
        sum = fmaf(l[i], m[i], sum);
      }
      float f = 0.f;
      if (h < nh)
        f = softmax_factor(top, sum, p.sink, h0 + h,
                           p.lse != nullptr && share == 0 ? p.lse + static_cast<int64_t>(t) * H + h0 + h : nullptr);
      for (int i = 0; i < shares; ++i) join_s[i * kTcAttnHeads + h] = m[i] * f;
    }
    __syncthreads();
    // this CTA's dims, four heads at a time
    const int per = D / shares;
    uint16_t* out = p.out + (static_cast<int64_t>(t) * H + h0) * D;
    for (int i = threadIdx.x; i < per * 16; i += kTcAttnThreads) {
      const int d = share * per + i % per;
      const int uu = i / per;
      if (4 * uu >= nh) continue;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < shares; ++k) {
        const float4 v = ld_cluster_f4(smem_addr(kv_s) + join_at(d, uu) * 16, k);
        const float4 f = *reinterpret_cast<const float4*>(join_s + k * kTcAttnHeads + 4 * uu);
        acc[0] = fmaf(v.x, f.x, acc[0]);
        acc[1] = fmaf(v.y, f.y, acc[1]);
        acc[2] = fmaf(v.z, f.z, acc[2]);
        acc[3] = fmaf(v.w, f.w, acc[3]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * uu + j < nh) {
          const __nv_bfloat16 ob = __float2bfloat16_rn(acc[j]);
          out[static_cast<int64_t>(4 * uu + j) * D + d] = *reinterpret_cast<const uint16_t*>(&ob);
        }
    }
    cluster_sync_all();  // no CTA leaves while another reads its partial outputs
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tbase, L::kTmemCols);
}

}  // namespace dsa
