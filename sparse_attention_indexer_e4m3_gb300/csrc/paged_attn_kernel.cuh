// Attention of each token over the rows of its sequence in a bf16 paged cache, on the tensor cores.  Token t at
// position p of sequence r sees the rows j <= p, of which with a window W only j > p - W, and j < F.  For head h
//     x_j = scale * q[t,h,:] . kv_j,   out[t,h,:] = sum_j e^{x_j} kv_j / ( sum_j e^{x_j} + e^{sink[h]} )
// (a kv row is both key and value).  Products run on bf16 operands with fp32 accumulators; the weights enter the second
// one as bf16 (off by half a step, 2^-8 of each, at most), the denominator sums them in fp32.
//
// Rows of q are (token, head) pairs, which lie one after the other; a unit is up to N of them.  Its tokens need not
// share a sequence: the unit's blocks are those of its runs of tokens of one sequence, one run after the other, and
// a run's blocks are masked for the other tokens.  (An instruction of N = 128 columns takes 64 cycles, one of 64 takes
// 48: idle columns cost little.)
//
// All blocks of all units, and for each unit a constant for its q and output, lie on one line that is cut into as
// many equal pieces as there are CTAs; each CTA finds its piece by a scan over the units.  So one long sequence
// uses all SMs, a batch of uneven ones keeps them equally busy, and a prompt's units go out whole but for one at
// each cut.  The parts of a unit that several CTAs share go to the workspace and are joined by a second kernel.
//
// One CTA per SM; per block of B rows (128; 64 at D = 512):
//   scout    (warp 2)      the unit's runs and blocks; the pages of the next blocks, four blocks at a time;
//   load     (last warps)  the rows by TMA into a ring of tiles of 128 dims, as chunks of [B rows x 128 bytes], 128-byte
//                          swizzled, page by page (a page without a row that some token sees becomes zeros: its
//                          memory is not read); the first of these warps brings q as well;
//   score    (warp 0)      the score product, K = D (tcgen05.mma kind::f16, bf16);
//   softmax  (warps 3-10)  weights as bf16; a running bound moves only when exceeded by more than 2^8, so the
//                          accumulators are rarely read back;
//   weighted (warp 1)      the weighted sum, K = B rows.
// Score products run ahead of the weighted sums by the places for scores, into the next unit as well.
//
// D <= 256: S = Q . KV^T, O += P . KV, with N = 128 rows of q in the lanes of tensor memory.  A softmax thread has a whole row:
// largest score and sum need no other thread, and the weights go back into tensor memory over the scores, from
// where the second product takes them.  Two groups of four warps take turns, so one block's exponentials run beside the next
// one's.  D = 512: the accumulators of 128 rows would fill tensor memory, so S^T = KV . Q^T and O^T += KV^T . P^T with 64
// rows of q as columns, P through shared memory, and a thread with one kv row of the block and 16 columns.  (As columns at
// D <= 256, too, a prompt with a window took 643 us instead of 278, drafts 208 instead of 77.)
//
// What bounds it (times at the sizes given, GB300):
//   - a batch of long sequences: reading them.  64 sequences of up to 65536 rows of 512, 64 heads: 367 to 384 us, 6.7 TB/s and
//     more, what a copy reaches (a part stays in L2).
//   - prompts at D = 512: the products.  Their operands come from shared memory at 128 bytes a clock, (M + N) / 4 cycles an
//     instruction: 48 for M = 128, N = 64, 34 for M = 64; 1872 of the 2070 cycles of a block of 64 rows.  4096 tokens over 8192 rows,
//     64 heads: 2.92 ms, 1130 TFLOP/s.
//   - prompts and drafts at D <= 256: the places for scores.  One is taken from its score product (1000 cycles behind the
//     products before it) over the softmax (2200) to the end of its weighted sum (1000), three of them turn over a block in 1500
//     cycles where the products need 1024; blocks that not every row sees all of take 1800 longer, and a unit's end and beginning
//     some 7000.  2700-token prompts with a window of 1024 at D = 128, 32 heads: 187 us.
//   - single tokens: a chain of launch, plan, table, rows, two products, some 128 partial outputs through L2 (as many bytes as the
//     rows) and the join.  One token over 32768 rows of 512, 64 heads: 22.3 us.
// Measured and slower at D <= 256: sixteen softmax warps with half a row each (191 us for 187; window decode 24.5 for
// 23.5), masks and outputs 32 rows or dims at a time (195 to 275 us), a place of its own for P (216).
#pragma once

#include <cuda_bf16.h>

#include "attn_kv4_kernel.cuh"
#include "kv4_codec_kernel.cuh"
#include "paged.cuh"
#include "tile_ring.h"

namespace dsa {

constexpr int kPgFirstSoft = 3;           // first softmax warp: the three before issue the two products, and scout
constexpr int kPgSoftWarps = 8;
constexpr int kPgSoft = 32 * kPgSoftWarps;
constexpr int kPgFirstLoad = kPgFirstSoft + kPgSoftWarps;  // first loading warp
constexpr int kPgSlots = 8;               // blocks whose pages are looked up ahead
constexpr int kPgBatch = 4;               // blocks looked up at a time
constexpr int kPgMaxTokens = 32;          // tokens of a unit: a lane of the scout each
constexpr float kPgNoBound = -3e38f;      // bound of a column without rows so far

// Columns of a unit at head dimension D (with 128 the output accumulators of D = 512 would take all tensor memory), and
// rows of a block.
__host__ __device__ constexpr int paged_cols(int D) { return D == 512 ? 64 : 128; }
__host__ __device__ constexpr int paged_block(int D) { return D == 512 ? 64 : 128; }
// What a unit costs beside its blocks, and the least piece of the line of a CTA (joining a part takes about as long), in blocks.
// (A cost of 1: drafts 72 us, window decode 27, window prompt 200; 4: 63 to 67, 24, 188; 8: 67, 23, 188.  Least pieces of 1:
// one token 23.2 us; these: 22.5; twice these: 25.2.)
constexpr int kPgUnitCost = 4;
__host__ __device__ constexpr int paged_min_piece(int D) { return D == 512 ? 4 : 2; }

// What the load and softmax warps know of a block.
struct PagedBlock {
  int row;         // its first row in the sequence
  int i0, i1;      // tokens of the unit that it is for
  int full;        // every column sees every row
  int starts;      // the first block of its tokens here
  uint32_t pages;  // bit i: page i of the block is there
  int id[8];       // pages of the block
  int tail;        // rows from this on nobody sees (they may never have been written)
  int pad[1];
};

// What the CTA does of a unit.
struct PagedPart {
  int unit;
  int blocks;   // of this CTA
  int way;      // kPgWhole: the CTA has all blocks; kPgHead: the first ones; kPgTail: later ones
  int row0;     // the unit's rows of q, and the rows of its first token before them
  int cols;
  int skip;
  int pad[2];
};
constexpr int kPgWhole = 0, kPgHead = 1, kPgTail = 2;

template <int D>
struct PagedLayout {
  static constexpr bool kByRow = D <= 256;                           // a softmax thread has a row of q (else a row of the block)
  static constexpr int kCols = paged_cols(D);
  static constexpr int kKeys = paged_block(D);
  static constexpr int kLoaders = D == 512 ? 4 : 1;                  // loading warps: every kLoaders-th tile is one's
  static constexpr int kThreads = 32 * (kPgFirstLoad + kLoaders);
  static constexpr int kChunks = D / 64;
  static constexpr int kTiles = D >= 128 ? D / 128 : 1;              // tiles of a block
  static constexpr int kTileChunks = kChunks / kTiles;
  static constexpr int kChunkBytes = kKeys * 128;
  static constexpr int kTileBytes = kTileChunks * kChunkBytes;
  static constexpr int kRing = D == 512 ? 9 : (D == 64 ? 8 : 5);     // tiles held
  static constexpr int kQBufs = D <= 128 ? 2 : 1;
  static constexpr int kQChunkBytes = kCols * 128;
  static constexpr int kQBytes = kChunks * kQChunkBytes;
  static constexpr int kKv = 0;
  static constexpr int kQ = kKv + kRing * kTileBytes;
  static constexpr int kP = kQ + kQBufs * kQBytes;                // not by row: two of bf16 [rows][64 columns]
  static constexpr int kNeg = kP + (kByRow ? 0 : 2 * kKeys * kCols * 2);  // float [cols] the running bounds (log2 units); not by row: negated
  static constexpr int kAlpha = kNeg + kCols * 4;                 // float [cols] rescale / output factors; by row: [2][cols] sums
  static constexpr int kTop = kAlpha + (kByRow ? 2 : 1) * kCols * 4;  // not by row: int [cols] largest scores, being reduced
  static constexpr int kEnd = kTop + (kByRow ? 0 : 1) * kCols * 4;    // int [2][tokens] by unit: rows below this are seen
  static constexpr int kBlocks = kEnd + 2 * kPgMaxTokens * 4;     // PagedBlock [slots]
  static constexpr int kParts = kBlocks + kPgSlots * static_cast<int>(sizeof(PagedBlock));  // PagedPart [2]
  static constexpr int kPlan = kParts + 2 * static_cast<int>(sizeof(PagedPart));            // int [8]
  static constexpr int kScan = kPlan + 32;                        // int64 [warps]
  static constexpr int kBar = kScan + (kThreads / 32 + 1) / 2 * 16;
  static constexpr int kNumBars = 28 + 2 * kPgSlots + 2 * kRing;
  static constexpr int kSmem = kBar + kNumBars * 8;
  // softmax warps that read a block, or fill a P
  static constexpr int kReaders = kByRow ? kPgSoftWarps / 2 : kPgSoftWarps;
  // tensor memory: S (or S^T) of some blocks from column 0, O (or O^T) tile m behind them
  static constexpr int kScores = D <= 128 ? 3 : 2;
  static constexpr int kSCols = kByRow ? kKeys : kCols;
  static constexpr int kOTile = kByRow ? (D < 128 ? D : 128) : kCols;
  static_assert(kScores * kSCols + kTiles * kOTile <= 512, "tensor memory");
  static_assert(kRing >= kScores * kTiles, "the score products go ahead of the weighted sums");
  static_assert(kSmem <= 232448, "shared memory");
};
static_assert(sizeof(PagedBlock) == 64 && sizeof(PagedPart) == 32, "layout");

// mbar_wait with its loop out of line (written out at each of the kernel's waits it made 90 KB of code, and instructions were
// waited for), and the timer, which takes some hundred cycles to read, only after some rounds.
__device__ __noinline__ bool paged_wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err, int site) {
  uint64_t since = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    const uint64_t now = global_timer_ns();
    if (since == 0) since = now;
    if (now - since > kWaitLimitNs) {
      record_timeout(err, site);
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool paged_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned* err, int site) {
  return mbar_try_wait(bar, parity) || paged_wait_long(bar, parity, abort, err, site);
}

// ------------------------------------------------------------------------------------ units and runs

// Entries of the shared units in the workspace: one for each unit of either cut, or for each CTA where these are fewer.
__host__ __device__ __forceinline__ int paged_entries(const PagedAttnParams& p, int ctas) {
  const int units = p.whole.units > p.any.units ? p.whole.units : p.any.units;
  return units < ctas ? units : ctas;
}

constexpr int kPgCount = 4;  // places of a thread that the choice of the cut looks at

struct PagedUnit {
  int row0, cols;  // its (token, head) rows
  int t0, n;       // tokens that they lie in
  int skip;        // rows of the first token before them
};

// Unit u of the cut `any` or of `whole`.
__device__ __forceinline__ PagedUnit paged_unit(const PagedAttnParams& p, bool any, int u) {
  const int rows = any ? p.any.rows : p.whole.rows, groups = any ? 1 : p.whole.groups;
  PagedUnit r;
  if (groups > 1) {
    const int t = u / groups, h = (u % groups) * rows;
    r.row0 = t * p.H + h;
    r.cols = min(rows, p.H - h);
  } else {
    r.row0 = u * rows;
    r.cols = min(rows, p.T * p.H - r.row0);
  }
  r.t0 = p.by_H(r.row0);
  r.n = p.by_H(r.row0 + r.cols - 1) - r.t0 + 1;
  r.skip = r.row0 - r.t0 * p.H;
  return r;
}

// Sequence of token t (-1: none) and the end of what it sees (0: nothing).
__device__ __forceinline__ void paged_token(const PagedAttnParams& p, int t, int& seq, int& end) {
  seq = ld_after_wait(p.seq + t);
  const int pos = ld_after_wait(p.pos + t);
  const bool some = static_cast<unsigned>(seq) < static_cast<unsigned>(p.pages.R) && pos >= 0;
  seq = some ? seq : -1;
  end = some ? min(pos, INT32_MAX - 1) + 1 : 0;
}

// A run of tokens of one sequence, from what its tokens see: [0, some) and [low, high).
struct PagedRun {
  int low, high, some;
  __device__ __forceinline__ void start() {
    low = INT32_MAX;
    high = some = 0;
  }
  __device__ __forceinline__ void add(const PagedAttnParams& p, int end) {
    low = min(low, max(0, end - p.window));
    high = max(high, end);
    some = max(some, min(p.first, end));
  }
  // blocks [0, a) and [b, b + the rest); the number of them
  __device__ __forceinline__ int blocks(const PagedAttnParams& p, int size, int& a, int& b) const {
    const int rows = min(high, p.pages.M << p.pages.log_rows);
    const auto up_to = [&](int n) { return n > 0 ? (n - 1) / size + 1 : 0; };
    b = low / size;
    a = min(up_to(min(some, rows)), b);
    return a + max(0, up_to(rows) - b);
  }
};

// Blocks of a unit, by one thread (its tokens' sequences and positions are read four at a time).
__device__ __forceinline__ int paged_blocks(const PagedAttnParams& p, const PagedUnit& u, int size) {
  int n = 0, seq = -1, a, b;
  PagedRun run;
  run.start();
#pragma unroll 1
  for (int i0 = 0; i0 < u.n; i0 += 4) {
    int s[4], end[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = -1;
      end[i] = 0;
      if (i0 + i < u.n) paged_token(p, u.t0 + i0 + i, s[i], end[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s[i] != seq) {
        if (seq >= 0) n += run.blocks(p, size, a, b);
        run.start();
        seq = s[i];
      }
      if (s[i] >= 0) run.add(p, end[i]);
    }
  }
  return seq >= 0 ? n + run.blocks(p, size, a, b) : n;
}

// Factor of a column's outputs whose weights' bound is m (log2 units) and whose denominator is l, in units of 2^m,
// without the sink; writes the natural log of the whole denominator where lse is given (what is no number stays so, and a
// sink that is none makes it one).
__device__ __forceinline__ float paged_factor(float m, float l, const float* sink, int h, float* lse) {
  if (sink != nullptr) {
    const float s = ld_after_wait(sink + h);
    if (s != s) l = s;
  }
  if (l != l) {
    if (lse != nullptr) *lse = l;
    return l;
  }
  return softmax_factor(m, l, sink, h, lse);
}

// An fp32 value as an int of the same order.
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_ordered(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7FFFFFFF)); }

__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The largest of three values, no number where one of them is none.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// A value that is a number where all of 16 are.
__device__ __forceinline__ float any_nan(const float (&o)[16]) {
  float a = max3_nan(o[0], o[1], o[2]), b = max3_nan(o[3], o[4], o[5]);
#pragma unroll
  for (int j = 6; j < 14; j += 4) {
    a = max3_nan(a, o[j], o[j + 1]);
    b = max3_nan(b, o[j + 2], o[j + 3]);
  }
  return max3_nan(max3_nan(a, b, o[14]), o[15], o[15]);
}

// The low n bits (n in [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// Tensor-memory load of the 16 lanes that hold a quarter of an M = 64 accumulator: thread i has lane i % 16 and 16 columns, the
// upper half of the threads those 16 further on.
__device__ __forceinline__ void tmem_ld_half_x16(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16], 16;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Reduces n values a lane (one of each of n columns) across n lanes, by recursive halving: afterwards v[0] holds
// column lane % n.
template <int kN, class Op>
__device__ __forceinline__ void xpose_reduce(float (&v)[kN], int lane, Op op) {
#pragma unroll
  for (int half = kN / 2; half >= 1; half >>= 1) {
    const bool up = (lane & half) != 0;
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      if (i < half) {
        const float send = up ? v[i] : v[i + half];
        const float keep = up ? v[i + half] : v[i];
        v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, half));
      }
    }
  }
}

// tma_load_2d issued where `on` is set, by a warp whose operands are the same in all lanes (by lanes of their own, each with its
// operands, a copy took 200 cycles to issue).
__device__ __forceinline__ void tma_load_2d_if(uint32_t on, uint32_t smem_dst, const void* map, uint32_t bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(on)
      : "memory");
}

// mbar_arrive_expect_tx where `on` is set.
__device__ __forceinline__ void mbar_expect_if(uint32_t on, uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
               "r"(bytes), "r"(on)
               : "memory");
}

// Ties 32 destination registers of tensor-memory loads to the wait for them.
__device__ __forceinline__ void tmem_wait_ld_regs32(float* v) {
  tmem_wait_ld_regs16(v);
  uint32_t* r = reinterpret_cast<uint32_t*>(v + 16);
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// tcgen05.mma kind::f16 with the A operand in tensor memory, issued where `on` is set.
__device__ __forceinline__ void mma_f16_ts_if(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(on), "r"(acc)
      : "memory");
}

// Tensor-memory store of 16 columns of words.
__device__ __forceinline__ void tmem_st_words_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <int D>
__global__ void __launch_bounds__(PagedLayout<D>::kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
                      const PagedAttnParams p, unsigned* err) {
  using L = PagedLayout<D>;
  constexpr int N = L::kCols;
  constexpr int kKeys = L::kKeys;
  constexpr int kCh = L::kChunks;
  constexpr int kTi = L::kTiles;
  constexpr int kRing = L::kRing;
  constexpr int kQb = L::kQBufs;
  constexpr int kThreads = L::kThreads;
  extern __shared__ __align__(1024) uint8_t paged_smem[];
  uint8_t* smem = paged_smem;
  uint8_t* kv_s = smem + L::kKv;
  uint8_t* q_s = smem + L::kQ;
  uint8_t* p_s = smem + L::kP;
  float* neg_s = reinterpret_cast<float*>(smem + L::kNeg);
  float* alpha_s = reinterpret_cast<float*>(smem + L::kAlpha);
  int* top_s = reinterpret_cast<int*>(smem + L::kTop);
  int* end_s = reinterpret_cast<int*>(smem + L::kEnd);
  PagedBlock* block_s = reinterpret_cast<PagedBlock*>(smem + L::kBlocks);
  PagedPart* part_s = reinterpret_cast<PagedPart*>(smem + L::kParts);
  volatile int* plan_s = reinterpret_cast<volatile int*>(smem + L::kPlan);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bars + 0;      // [2]
  uint64_t* q_empty = bars + 2;     // [2]
  uint64_t* o_empty = bars + 6;
  uint64_t* drain = bars + 4;       // [2]
  uint64_t* part_full = bars + 8;   // [2]
  uint64_t* part_empty = bars + 10; // [2]
  uint64_t* s_full = bars + 12;     // [scores]
  uint64_t* p_full = bars + 25;     // [scores]
  uint64_t* decided = bars + 18;    // [4] by row: bounds of a quarter's rows
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 15);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* pv_done = bars + 22;    // [scores]
  uint64_t* blk_full = bars + 28;   // [slots]
  uint64_t* blk_empty = blk_full + kPgSlots;
  uint64_t* kv_full = blk_empty + kPgSlots;  // [ring]
  uint64_t* kv_empty = kv_full + kRing;

  if ((smem_addr(smem) & 1023u) != 0u) {  // (the swizzle goes by addresses; nothing else lies before this memory)
    wait_stream();
    if (threadIdx.x == 0) {
      record_error(err, kErrPlan);
      // (all CTAs are here: the join finds no shared unit, instead of what the workspace held)
      if (static_cast<int>(blockIdx.x) < paged_entries(p, static_cast<int>(gridDim.x))) p.shared[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x < kPgSlots * sizeof(PagedBlock) / 4) reinterpret_cast<int*>(block_s)[threadIdx.x] = 0;
  if (threadIdx.x < 2 * sizeof(PagedPart) / 4) reinterpret_cast<int*>(part_s)[threadIdx.x] = 0;
  if (!L::kByRow && threadIdx.x < N) top_s[threadIdx.x] = ordered(-INFINITY);
  if (threadIdx.x == 0) {
    mbar_init(o_empty, kPgSoftWarps);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&part_full[i], 1);
      mbar_init(&part_empty[i], 2 + L::kLoaders + kPgSoftWarps);
    }
    for (int i = 0; i < kPgSlots; ++i) {
      mbar_init(&blk_full[i], 1);
      mbar_init(&blk_empty[i], L::kLoaders + L::kReaders);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&decided[i], 1);
    for (int i = 0; i < L::kScores; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&pv_done[i], 1);
      mbar_init(&p_full[i], L::kReaders);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&kvmap);
    tma_prefetch_desc(&qmap);
  }
  fence_proxy_async_shared();
  wait_stream();  // (tensor memory is taken behind it: the kernel before may still have to allocate its own)
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }

  // ------------------------------------------------------------------ the CTA's piece of the line
  // Cost of a unit: its blocks and a constant.  [from, to) of the line is this CTA's.  A unit starts on one CTA's piece (which
  // has at least one of its blocks) and belongs to those, too, whose pieces its blocks reach into.
  constexpr int kUnitCost = kPgUnitCost;
  int64_t* warp_scan = reinterpret_cast<int64_t*>(smem + L::kScan);  // [warps]
  volatile uint32_t* issued_s = reinterpret_cast<volatile uint32_t*>(smem + L::kScan);  // later: tiles of each loading warp, and q's
  static_assert(4 * (L::kLoaders + 1) <= L::kBar - L::kScan, "counts in the scan's place");
  // Each unit's blocks, kept in the ring's place (where they fit: 32768 units are prompts of 65536 tokens and 64 heads).
  constexpr int kKeep = L::kQ / 4;
  int* blocks_s = reinterpret_cast<int*>(kv_s);
  // The cut: of these places (evenly spread ones where there are more) those with a token, and those whose next has one of the same
  // sequence.  (Read beside the blocks of the cut that is expected; the choice takes 0.7 of window decode's 24.7 us.)
  const bool choose = p.any.rows != p.whole.rows;
  const int looked = min(p.T, kPgCount * kThreads);
  int seq_of[kPgCount], seq_next[kPgCount];
#pragma unroll
  for (int i = 0; i < kPgCount; ++i) {
    seq_of[i] = seq_next[i] = -1;
    const int at = static_cast<int>(threadIdx.x) + i * kThreads;
    if (choose && at < looked) {
      const int t = looked == p.T ? at : static_cast<int>(static_cast<int64_t>(at) * p.T / looked);
      seq_of[i] = ld_after_wait(p.seq + t);
      if (t + 1 < p.T) seq_next[i] = ld_after_wait(p.seq + t + 1);
    }
  }
  bool any = p.guess != 0, keep;
  int units;
#pragma unroll 1
  for (bool chosen = !choose;; chosen = true) {
    units = any ? p.any.units : p.whole.units;
    keep = units <= kKeep;
    if (keep) {  // (each entry by the thread that wrote it before)
#pragma unroll 1
      for (int u = static_cast<int>(threadIdx.x); u < units; u += kThreads) blocks_s[u] = paged_blocks(p, paged_unit(p, any, u), kKeys);
    }
    int* count_s = end_s;  // [warps]
    static_assert(kThreads / 32 <= 2 * kPgMaxTokens && kPgCount * kThreads < 65536, "counts");
    int n = 0;  // tokens, and in the upper half those that are joined by the next
    if (!chosen) {
#pragma unroll
      for (int i = 0; i < kPgCount; ++i)
        if (static_cast<unsigned>(seq_of[i]) < static_cast<unsigned>(p.pages.R)) n += seq_next[i] == seq_of[i] ? 65537 : 1;
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) count_s[warp] = n;
    }
    __syncthreads();
    if (chosen) break;
    n = __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? count_s[lane] : 0);
    const int tokens = n & 0xFFFF, runs = tokens - (n >> 16);
    const bool better = p.per_token * static_cast<float>(tokens) + p.per_run * static_cast<float>(runs) < 0.f;  // (in all threads)
    if (better == any) break;
    any = better;
  }
  const auto blocks_of = [&](int u) { return keep ? blocks_s[u] : paged_blocks(p, paged_unit(p, any, u), kKeys); };
  const int u_first = static_cast<int>(static_cast<int64_t>(units) * threadIdx.x / kThreads);
  const int u_last = static_cast<int>(static_cast<int64_t>(units) * (threadIdx.x + 1) / kThreads);
  int64_t mine = 0;
#pragma unroll 1
  for (int u = u_first; u < u_last; ++u) mine += blocks_of(u) + kUnitCost;
  int64_t upto = mine;  // the line up to the end of this thread's units
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t other = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += other;
  }
  if (lane == 31) warp_scan[warp] = upto;
  __syncthreads();
  int64_t line = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t v = warp_scan[w];
    if (w < warp) upto += v;
    line += v;
  }
  const int64_t ctas = max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), line / paged_min_piece(D)));
  const int cta = static_cast<int>(blockIdx.x);
  const int64_t from = cta < ctas ? line * cta / ctas : line, to = cta < ctas ? line * (cta + 1) / ctas : line;
  if (from < to && mine > 0 && upto > from && upto - mine < to) {
    // the threads whose units the piece starts or ends on walk over them again
    int64_t at = upto - mine;
    if (at <= from || upto >= to) {
#pragma unroll 1
      for (int u = u_first; u < u_last; ++u) {
        const int nb = blocks_of(u);
        const int64_t next = at + nb + kUnitCost;
        if (at <= from && from < next) {
          plan_s[0] = u;
          plan_s[1] = static_cast<int>(min(from - at, static_cast<int64_t>(nb)));  // its first block here
          plan_s[2] = from == at;                                                    // it starts here
        }
        if (at < to && to <= next) {
          plan_s[3] = u;
          plan_s[4] = static_cast<int>(min(to - at, static_cast<int64_t>(nb)));  // the end of its blocks here
          // the last CTA that has one of its blocks: the one on whose piece the last of them lies
          plan_s[5] = static_cast<int>(((at + max(nb, 1)) * ctas - 1) / line);
          plan_s[6] = nb;
        }
        at = next;
      }
    }
  }
  fence_proxy_async_shared();  // (the copies write where the blocks were)
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const uint32_t s_tmem = tbase;
  const uint32_t o_tmem = tbase + L::kScores * L::kSCols;
  const bool idle = from >= to;
  const int unit0 = idle ? 0 : plan_s[0], unit1 = idle ? -1 : plan_s[3];
  const int from_block = plan_s[1], to_block = plan_s[4];
  const bool starts = plan_s[2] != 0;
  if (threadIdx.x == 0) {
    // entries of the shared units: by unit, written by the CTA that it starts on, where there are no more than CTAs, else by CTA
    const bool shared = !idle && to_block < plan_s[6] && (unit1 > unit0 || starts);
    int4 entry = make_int4(0, 0, 0, 0);
    if (shared) {
      const PagedUnit un = paged_unit(p, any, unit1);
      entry = make_int4(un.row0, cta, plan_s[5] - cta + 1, un.cols);
    }
    if (units > static_cast<int>(gridDim.x)) {
      p.shared[cta] = entry;
    } else {
      for (int u = starts ? unit0 : unit0 + 1; u <= unit1; ++u) p.shared[u] = u == unit1 ? entry : make_int4(0, 0, 0, 0);
    }
  }
  if (cta == 0)  // entries that the other cut would have
    for (int u = units + static_cast<int>(threadIdx.x); u < paged_entries(p, static_cast<int>(gridDim.x)); u += kThreads)
      p.shared[u] = make_int4(0, 0, 0, 0);
  const auto gone = [&]() -> bool { return __any_sync(0xffffffffu, *abort_flag != 0) != 0; };

  if (warp == 2) {
    // ------------------------------------------------------------------ scout
    uint32_t gb = 0;  // blocks of this CTA so far
    int n = 0;        // parts of this CTA so far
    constexpr int kPages = kKeys / 16;  // most pages of a block
    static_assert(kPages * kPgBatch <= 32, "a lane for each page of a batch");
    int seq = -1, end = 0;  // of the unit's token `lane`, read a unit ahead
    if (unit0 <= unit1) {
      const PagedUnit un = paged_unit(p, any, unit0);
      if (lane < un.n) paged_token(p, un.t0 + lane, seq, end);
    }
    bool ok = true;
    for (int u = unit0; ok && u <= unit1; ++u) {
      const PagedUnit un = paged_unit(p, any, u);
      const int my_seq = seq, my_end = end;
      seq = -1;
      end = 0;
      if (u < unit1) {
        const PagedUnit next = paged_unit(p, any, u + 1);
        if (lane < next.n) paged_token(p, next.t0 + lane, seq, end);
      }
      // tokens that begin a run, and the runs' spans: reduced over their lanes
      const int before_seq = __shfl_up_sync(0xffffffffu, my_seq, 1);
      const uint32_t begins = __ballot_sync(0xffffffffu, lane < un.n && (lane == 0 || my_seq != before_seq));
      const auto run_of = [&](int i0, int i1) {
        const bool in = lane >= i0 && lane < i1;
        PagedRun run;
        run.low = __reduce_min_sync(0xffffffffu, in ? max(0, my_end - p.window) : INT32_MAX);
        run.high = __reduce_max_sync(0xffffffffu, in ? my_end : 0);
        run.some = __reduce_max_sync(0xffffffffu, in ? min(p.first, my_end) : 0);
        return run;
      };
      const auto run_end = [&](int i0) {
        const uint32_t after = i0 < 31 ? begins & ~low_bits(i0 + 1) : 0u;
        return after != 0u ? __ffs(after) - 1 : un.n;
      };
      int nb = 0;
      for (int i = 0; i < un.n;) {
        const int i1 = run_end(i);
        int a, b;
        if (__shfl_sync(0xffffffffu, my_seq, i) >= 0) nb += run_of(i, i1).blocks(p, kKeys, a, b);
        i = i1;
      }
      const int b0 = u == unit0 ? from_block : 0, b1 = u == unit1 ? to_block : nb;
      const int way = u == unit0 && !starts ? kPgTail : (b1 < nb ? kPgHead : kPgWhole);
      if (way == kPgTail && b0 >= b1) continue;  // (its blocks end before this CTA's piece)
      if (n > 1) paged_wait(&part_empty[n & 1], static_cast<uint32_t>((n >> 1) - 1) & 1u, abort_flag, err, 0x80);
      if (gone()) break;
      end_s[(n & 1) * kPgMaxTokens + lane] = my_end;
      if (lane == 0) {
        part_s[n & 1].unit = u;
        part_s[n & 1].blocks = b1 - b0;
        part_s[n & 1].way = way;
        part_s[n & 1].row0 = un.row0;
        part_s[n & 1].cols = un.cols;
        part_s[n & 1].skip = un.skip;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&part_full[n & 1]);
      ++n;
      int before = 0;  // blocks of the runs before
      for (int i0 = 0; ok && i0 < un.n && before < b1;) {
        const int i1 = run_end(i0), s = __shfl_sync(0xffffffffu, my_seq, i0);
        const int first_token = i0;
        i0 = i1;
        if (s < 0) continue;
        const PagedRun run = run_of(first_token, i1);
        int ra, rb;
        const int count = run.blocks(p, kKeys, ra, rb);
        const bool in = lane >= first_token && lane < i1;
        const int all_low = __reduce_max_sync(0xffffffffu, in ? max(0, my_end - p.window) : 0);
        const int all_end = __reduce_min_sync(0xffffffffu, in ? my_end : INT32_MAX);
        const bool whole = first_token == 0 && i1 == un.n;
        const int32_t* table = p.pages.table + static_cast<int64_t>(s) * p.pages.M;
        const int k_first = max(0, b0 - before), k_end = min(count, b1 - before);
        // lane = (block of the batch, page of the block)
        const int sub = lane & 7, off = sub << p.pages.log_rows;
        const bool is_page = sub < kPages && off < kKeys;
        const uint32_t want = __ballot_sync(0xffffffffu, is_page) & 0xFFu;
        const auto first_row = [&](int k0) {
          const int k = min(k0 + (lane >> 3), k_end - 1);
          return (k < ra ? k : rb + k - ra) * kKeys;
        };
        const int span = min(1 << p.pages.log_rows, kKeys);
        const auto look_up = [&](int k0) -> int {  // -1: no page, or none of whose rows [at, at + span) some token of the run sees
          if (k0 >= k_end) return -1;
          const int at = first_row(k0) + off, index = at >> p.pages.log_rows;
          const bool there = is_page && (at < run.some || (at < run.high && at - run.low > -span));
          int page = -1;
          if (there && index < p.pages.M) page = ld_after_wait(table + index);
          return page;
        };
        int next_page = k_first < k_end ? look_up(k_first) : -1;
        for (int k0 = k_first; ok && k0 < k_end; k0 += kPgBatch) {
          int page = next_page;
          next_page = look_up(k0 + kPgBatch);  // (in flight while this batch is handed out)
          const int row = first_row(k0);
          if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages.P)) page = -1;
          const uint32_t mapped = __ballot_sync(0xffffffffu, page >= 0);
          for (int j = 0; j < kPgBatch && k0 + j < k_end; ++j, ++gb) {
            const uint32_t slot = gb % kPgSlots;
            if (gb >= kPgSlots) paged_wait(&blk_empty[slot], (gb / kPgSlots - 1) & 1u, abort_flag, err, 0x81);
            if (gone()) {
              ok = false;
              break;
            }
            PagedBlock& blk = block_s[slot];
            if ((lane >> 3) == j) blk.id[sub] = page;
            if (lane == 8 * j) {
              const uint32_t have = (mapped >> (8 * j)) & 0xFFu;
              blk.row = row;
              blk.i0 = first_token;
              blk.i1 = i1;
              blk.pages = have;
              blk.starts = k0 + j == k_first;
              blk.tail = min(run.high - row, kKeys);
              blk.full = whole && have == want && row <= all_end - kKeys && (row >= all_low || row <= p.first - kKeys);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&blk_full[slot]);
          }
        }
        before += count;
      }
    }
    // the end: a part without a unit
    if (!gone()) {
      if (n > 1) paged_wait(&part_empty[n & 1], static_cast<uint32_t>((n >> 1) - 1) & 1u, abort_flag, err, 0x82);
      if (!gone() && lane == 0) {
        part_s[n & 1].unit = -1;
        part_s[n & 1].blocks = 0;
        mbar_arrive(&part_full[n & 1]);
      }
    }
  } else if (warp >= kPgFirstLoad) {
    // ------------------------------------------------------------------ load (warps that elect a thread)
    const uint32_t on = elect_one();
    const int loader = warp - kPgFirstLoad;  // its tiles: loader, loader + kLoaders, ...; q is the first one's
    const auto wait = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
      return __all_sync(0xffffffffu, paged_wait(bar, parity, abort_flag, err, site)) != 0;
    };
    uint32_t gb = 0, nq = 0;                                          // blocks and q's of this CTA so far
    TileRing<kRing, L::kLoaders> ring(static_cast<uint32_t>(loader));  // its tiles
    const int page_rows = 1 << p.pages.log_rows;
    const int boxes = kKeys / p.box_rows;                    // copies of a block and chunk
    const int none = max(1, p.pages.P << p.pages.log_rows);  // a row behind the last page: the copy fills in zeros
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!wait(&part_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, 0x83)) break;
      const int u = __reduce_max_sync(0xffffffffu, part_s[n & 1].unit);
      const int nb = __reduce_max_sync(0xffffffffu, part_s[n & 1].blocks);
      const int y = __reduce_max_sync(0xffffffffu, part_s[n & 1].row0);
      if (lane == 0) mbar_arrive(&part_empty[n & 1]);
      __syncwarp();
      if (u < 0) break;
      if (loader == 0 && nb > 0) {
        // a place for q is free once the score products of the part that had it are done
        const uint32_t qb = nq % kQb;
        if (nq >= kQb && !wait(&q_empty[qb], (nq / kQb - 1) & 1u, 0x84)) break;
        ++nq;
        const uint32_t bar = smem_addr(&q_full[qb]), to = smem_addr(q_s) + qb * L::kQBytes;
        mbar_expect_if(on, bar, L::kQBytes);
#pragma unroll
        for (int c = 0; c < kCh; ++c) tma_load_2d_if(on, to + c * L::kQChunkBytes, &qmap, bar, 64 * c, y);
      }
      for (int b = 0; ok && b < nb; ++b, ++gb) {
        const uint32_t slot = gb % kPgSlots;
        if (!wait(&blk_full[slot], (gb / kPgSlots) & 1u, 0x85)) {
          ok = false;
          break;
        }
        // the row of the pages of the lane's box
        const int from = lane % 8 * p.box_rows, page = block_s[slot].id[(from >> p.pages.log_rows) & 7];
        const int mine = page >= 0 ? (page << p.pages.log_rows) + ((block_s[slot].row + from) & (page_rows - 1)) : none;
        __syncwarp();
        if (lane == 0) mbar_arrive(&blk_empty[slot]);
#pragma unroll
        for (int m0 = 0; m0 < kTi; m0 += L::kLoaders) {
          if (ring.round > 0 && !wait(&kv_empty[ring.at], (ring.round - 1) & 1u, 0x86)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_addr(&kv_full[ring.at]);
          uint32_t to = smem_addr(kv_s) + ring.at * L::kTileBytes;
          mbar_expect_if(on, bar, L::kTileBytes);
#pragma unroll 1
          for (int i = 0; i < boxes; ++i, to += p.box_rows * 128) {
            const int y = __shfl_sync(0xffffffffu, mine, i);
#pragma unroll
            for (int c = 0; c < L::kTileChunks; ++c)
              tma_load_2d_if(on, to + c * L::kChunkBytes, &kvmap, bar, 64 * (L::kTileChunks * (m0 + loader) + c), y);
          }
          ring.next();
        }
      }
    }
    if (lane == 0) {
      issued_s[loader] = ring.issued;
      if (loader == 0) issued_s[L::kLoaders] = nq;
    }
  } else if (warp < 2) {
    // ------------------------------------------------------------------ MMA issuers (whole warps, one thread of each elected)
    // Warp 0 issues the score products, as the rows and a place for the scores come in, warp 1 the weighted sums, as the
    // weights do: neither waits for what the other needs, and their loops are short.
    const uint32_t on = elect_one();
    const auto wait = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
      return __all_sync(0xffffffffu, paged_wait(bar, parity, abort_flag, err, site)) != 0;
    };
    // A value of the warp by a reduction, whose result the compiler knows to be the same for all lanes: so addresses and
    // descriptors stay in uniform registers (without it an instruction took 80 cycles to issue, longer than to run).
    const auto uniform = [](uint32_t v) { return __reduce_max_sync(0xffffffffu, v); };
    // by row: S = Q . KV^T and O += P . KV with P in tensor memory; else S^T = KV . Q^T and O^T += KV^T . P^T
    constexpr uint32_t id_qk = L::kByRow ? idesc_bf16(N, kKeys, false, false) : idesc_bf16(kKeys, N, false, false);
    constexpr uint32_t id_pv = L::kByRow ? idesc_bf16(N, L::kOTile, false, true) : idesc_bf16(128, N, true, true);
    const uint64_t kv_k = desc_sw128(smem_addr(kv_s), 16, 1024);                // K-major: rows x dims
    const uint64_t q_k = desc_sw128(smem_addr(q_s), 16, 1024);                  // K-major: columns x dims
    const uint64_t kv_mn = desc_sw128(smem_addr(kv_s), L::kChunkBytes, 1024);   // MN-major: dims x rows
    const uint64_t p_mn = desc_sw128(smem_addr(p_s), kKeys * 128, 1024);        // MN-major: columns x rows
    uint32_t gb = 0, parts = 0, nq = 0;  // blocks, units and q's so far
    uint32_t at = 0, round = 0;          // the next tile's place in the ring, and how often it was used before
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!wait(&part_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, 0x90)) break;
      const int u = __reduce_max_sync(0xffffffffu, part_s[n & 1].unit);
      const int nb = __reduce_max_sync(0xffffffffu, part_s[n & 1].blocks);
      if (lane == 0) mbar_arrive(&part_empty[n & 1]);
      __syncwarp();
      if (u < 0) break;
      ++parts;
      if (nb == 0) continue;
      if (warp == 0) {
        const uint32_t qb = nq % kQb;
        if (!wait(&q_full[qb], (nq / kQb) & 1u, 0x91)) break;
        ++nq;
        const uint64_t q = q_k + uniform(qb * (L::kQBytes >> 4));
        for (int b = 0; ok && b < nb; ++b, ++gb) {
          // a place for the scores: by row, where the weights of the block before in it were summed; else, where they were formed
          if (gb >= L::kScores &&
              !wait(&(L::kByRow ? pv_done : p_full)[gb % L::kScores], (gb / L::kScores - 1) & 1u, 0x92)) {
            ok = false;
            break;
          }
          const uint32_t to = uniform(s_tmem + L::kSCols * (gb % L::kScores));
#pragma unroll
          for (int m = 0; m < kTi; ++m) {
            if (!wait(&kv_full[at], round & 1u, 0x93)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint64_t a = kv_k + uniform(at * (L::kTileBytes >> 4));
            if (++at == kRing) {
              at = 0;
              ++round;
            }
#pragma unroll
            for (int k = 0; k < 4 * L::kTileChunks; ++k) {
              const uint64_t kv = a + (((k / 4) * L::kChunkBytes + (k % 4) * 32) >> 4);
              const uint64_t qd = q + (((m * L::kTileChunks + k / 4) * L::kQChunkBytes + (k % 4) * 32) >> 4);
              if (m == 0 && k == 0)
                mma_f16_if<false>(on, to, L::kByRow ? qd : kv, L::kByRow ? kv : qd, id_qk, 0u);
              else
                mma_f16_if<true>(on, to, L::kByRow ? qd : kv, L::kByRow ? kv : qd, id_qk);
            }
          }
          if (!ok) break;
          mma_commit_if(on, &s_full[gb % L::kScores]);
        }
        if (ok) mma_commit_if(on, &q_empty[qb]);  // (after the part's last score product)
      } else {
        for (int b = 0; ok && b < nb; ++b, ++gb) {
          // (a part's first weighted sum overwrites O: the output of the part before must be read)
          if (!wait(&p_full[gb % L::kScores], (gb / L::kScores) & 1u, 0x94) || (b == 0 && parts > 1 && !wait(o_empty, parts & 1u, 0x95))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t weights_at = uniform(s_tmem + L::kSCols * (gb % L::kScores));   // by row
          const uint64_t weights = p_mn + uniform((gb & 1u) * (kKeys * 128 >> 4));       // not by row
#pragma unroll
          for (int m = 0; m < kTi; ++m) {
            const uint64_t a = kv_mn + uniform(at * (L::kTileBytes >> 4));
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ++ks) {
              const uint64_t kv = a + ((ks * 16 * 128) >> 4);
              if constexpr (L::kByRow)
                mma_f16_ts_if(on, o_tmem + L::kOTile * m, weights_at + 8 * ks, kv, id_pv, b > 0 || ks > 0 ? 1u : 0u);
              else if (ks == 0)
                mma_f16_if<false>(on, o_tmem + L::kOTile * m, kv, weights + ((ks * 16 * 128) >> 4), id_pv, b > 0 ? 1u : 0u);
              else
                mma_f16_if<true>(on, o_tmem + L::kOTile * m, kv, weights + ((ks * 16 * 128) >> 4), id_pv);
            }
            mma_commit_if(on, &kv_empty[at]);
            if (++at == kRing) at = 0;
          }
          mma_commit_if(on, &pv_done[gb % L::kScores]);
        }
      }
    }
    // every MMA issued by this thread has completed once `drain` flips
    mma_commit_if(on, &drain[warp]);
    mbar_wait_drain(&drain[warp], 0);
    __syncwarp();
  } else if constexpr (L::kByRow) {
    // ------------------------------------------------------------------ softmax and output, a thread with a row of q
    // Warps 3-6 take the even blocks, 7-10 the odd ones; a row's two threads (of the same quarter of the two groups) take
    // turns in deciding on its bound, so a block's exponentials run beside the next one's.  The hardware barriers, whose wait
    // has no limit, are those of a unit, which all pass or none: a block has none.
    const int group = (warp - kPgFirstSoft) >> 2;
    const int quarter = warp & 3;               // tensor-memory lane quarter
    const int r = quarter * 32 + lane;          // the unit's row
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float to_log2 = p.to_log2[0];
    const uint64_t to_log2_2 = *reinterpret_cast<const uint64_t*>(p.to_log2);
    volatile float* bound_s = neg_s;                                  // [N]
    float* sum_s = alpha_s;                                           // [2][N]
    uint32_t gb0 = 0;                                                 // blocks of the parts before
    float x[kKeys];                                                   // the row's scores, exponents, weights
    for (int n = 0;; ++n) {
      paged_wait(&part_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, err, 0xA0);
      const int nb = part_s[n & 1].blocks;
      if (bar_or(kTcEpiBar, kPgSoft, *abort_flag != 0)) break;
      if (part_s[n & 1].unit < 0) break;
      const bool used = quarter * 32 < part_s[n & 1].cols;  // (of a quarter without rows nothing is read, written or kept)
      float l0 = 0.f, l_bound = kPgNoBound;                 // this thread's sum, in units of 2^l_bound
      for (int b = static_cast<int>(gb0 + ((gb0 ^ group) & 1u)); static_cast<uint32_t>(b) < gb0 + nb; b += 2) {  // (of all blocks so far)
        const uint32_t gb = static_cast<uint32_t>(b), slot = gb % kPgSlots;
        paged_wait(&blk_full[slot], (gb / kPgSlots) & 1u, abort_flag, err, 0xA1);
        const PagedBlock& blk = block_s[slot];
        const int row = blk.row;
        const bool full = __any_sync(0xffffffffu, blk.full != 0) != 0;
        const int i0 = blk.i0, i1 = blk.i1;
        const uint32_t there = blk.pages;
        const int tail = blk.tail;
        __syncwarp();
        if (lane == 0) mbar_arrive(&blk_empty[slot]);
        bool mine = false;  // its token is one of the block's
        int end = 0, low = 0;
        if (!full && r < part_s[n & 1].cols) {
          const int token = p.by_H(part_s[n & 1].skip + r);
          mine = token >= i0 && token < i1;
          end = end_s[(n & 1) * kPgMaxTokens + token];
          low = max(0, end - p.window);
        }
        // The block's rows [32 i, 32 i + 32) that this row sees.
        const auto mask_of = [&](int i) -> uint32_t {
          if (!mine) return 0u;
          const auto upto = [&](int e) { return low_bits(min(max(e - row - 32 * i, 0), 32)); };
          uint32_t m = upto(end) & (~upto(low) | upto(p.first));
          if (p.pages.log_rows == 4) {  // two pages
            if (((there >> (2 * i)) & 1u) == 0u) m &= 0xFFFF0000u;
            if (((there >> (2 * i + 1)) & 1u) == 0u) m &= 0x0000FFFFu;
          } else if (((there >> ((32 * i) >> p.pages.log_rows)) & 1u) == 0u) {
            m = 0u;
          }
          return m;
        };
        const uint32_t s_at = s_tmem + L::kSCols * (gb % L::kScores) + lane_off;
        paged_wait(&s_full[gb % L::kScores], (gb / L::kScores) & 1u, abort_flag, err, 0xA2);
        tc_fence_after_sync();
        if (tail < kKeys) {  // rows that may never have been written: weights of 0 times what is no number would be none
          for (int c = 0; c < kCh; ++c) {
            const uint32_t tile = gb * kTi + c / L::kTileChunks;
            uint8_t* chunk = kv_s + (tile % kRing) * L::kTileBytes + (c % L::kTileChunks) * L::kChunkBytes;
            for (int i = tail * 128 + ((warp - kPgFirstSoft) & 3) * 512 + lane * 16; i < L::kChunkBytes; i += 2048)
              *reinterpret_cast<uint4*>(chunk + i) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_shared();
        }
        // the largest score
        float top = -INFINITY;
        if (used) {
#pragma unroll
          for (int i = 0; i < kKeys; i += 32) tmem_ld_x32(s_at + i, x + i);
#pragma unroll
          for (int i = 0; i < kKeys; i += 32) tmem_wait_ld_regs32(x + i);
          if (!full) {
            if (tail < kKeys) {
#pragma unroll
              for (int c = 0; c < kKeys; ++c)
                if (c >= tail) x[c] = 0.f;
            }
            uint64_t none = 0ull;  // is a number where every score is
#pragma unroll
            for (int c = 0; c < kKeys; c += 2) none = fma_f32x2(pack_f32x2(x[c], x[c + 1]), 0ull, none);
            float n0, n1;
            unpack_f32x2(none, n0, n1);
            if (__any_sync(0xffffffffu, mine && (n0 != n0 || n1 != n1))) {
              // Weights of 0 times values that are no numbers would still be none.  So the kv rows that hold such are taken out (by each
              // warp with rows of q of the block's tokens: all of those find them), and rows of q that see one get a sum that is
              // none.  What was taken out is -0 all over, so that a warp that comes later finds it as well: where another is at it, each
              // word that held one either still does or is a pair of -0.  (A row that holds such a pair of its own is not written, and
              // counts only where its score overflows.)  Scores of other rows of q show nothing: these may hold anything.  (Four tokens
              // over 20000 rows beside four places with q that is none, D = 128: 47 us with their scores looked at, 20.5 without.)
              constexpr uint32_t kOut = 0x80008000u;
              bool sees = false;
#pragma unroll 1
              for (int i = 0; i < kKeys; i += 16) {
                float y[16];
                tmem_ld_x16(s_at + i, y);
                tmem_wait_ld_regs16(y);
                uint32_t is = 0u;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  if (i + c < tail && !(fabsf(y[c]) < INFINITY)) is |= 1u << c;
                const uint32_t seen = is & (mask_of(i / 32) >> (i & 16));
                is = __reduce_or_sync(0xffffffffu, mine ? is : 0u);
                while (is != 0u) {
                  const int c = __ffs(is) - 1, key = i + c;
                  is &= is - 1u;
                  const auto at = [&](int j) -> uint4* {  // piece j of the row
                    const uint32_t tile = gb * kTi + (j / 8) / L::kTileChunks;
                    paged_wait(&kv_full[tile % kRing], (tile / kRing) & 1u, abort_flag, err, 0xA6);
                    const int chunk = static_cast<int>(tile % kRing) * L::kTileBytes + ((j / 8) % L::kTileChunks) * L::kChunkBytes;
                    return reinterpret_cast<uint4*>(kv_s + chunk + key * 128) + j % 8;
                  };
                  uint32_t found = 0u;  // bit 0: what is no number, bit 1: what was taken out
#pragma unroll 1
                  for (int j = lane; j < kCh * 8; j += 32) {
                    const uint4 v = *at(j);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      if (w[k] == kOut) found |= 2u;
                      if ((w[k] & 0x7F80u) == 0x7F80u || (w[k] & 0x7F800000u) == 0x7F800000u) found |= 1u;
                    }
                  }
                  found = __reduce_or_sync(0xffffffffu, found);
                  if ((found & 1u) != 0u) {
#pragma unroll 1
                    for (int j = lane; j < kCh * 8; j += 32) *at(j) = make_uint4(kOut, kOut, kOut, kOut);
                  }
                  sees |= found != 0u && ((seen >> c) & 1u) != 0u;
                }
              }
              if (sees) l0 = __int_as_float(0x7FFFFFFF);
              fence_proxy_async_shared();
            }
            const float hidden = to_log2 < 0.f ? INFINITY : -INFINITY;
#pragma unroll
            for (int i = 0; i < kKeys; i += 32) {
              const uint32_t mask = mask_of(i / 32);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if ((mask & (1u << c)) == 0u) x[i + c] = hidden;
            }
          }
          float t[4] = {x[0], x[1], x[2], x[3]};
          if (to_log2 < 0.f) {
#pragma unroll
            for (int c = 4; c < kKeys; ++c) t[c & 3] = fminf(t[c & 3], x[c]);
            top = -fminf(fminf(t[0], t[1]), fminf(t[2], t[3]));
          } else {
#pragma unroll
            for (int c = 4; c + 8 <= kKeys; c += 8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) t[k] = max3(t[k], x[c + k], x[c + 4 + k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = fmaxf(t[k], x[kKeys - 4 + k]);
            top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
          }
        }
        // the bound: raised only when exceeded by more than 2^8, behind the decision on the block before
        if (gb > 0) paged_wait(&decided[quarter], (gb - 1) & 1u, abort_flag, err, 0xA7);
        float before = kPgNoBound;
        if (gb != gb0) before = bound_s[r];
        float bound = before;
        const float most = top * fabsf(to_log2);
        if (most > before + kTcLazyLog2) bound = most;
        bound_s[r] = bound;
        __syncwarp();
        if (lane == 0) mbar_arrive(&decided[quarter]);
        const bool moved = bound != before && before != kPgNoBound;
        if (__any_sync(0xffffffffu, used && moved)) {  // the accumulators of the blocks before follow
          // (the last block's scores came behind the weighted sum kScores blocks before it, so the phase is the barrier's next)
          paged_wait(&pv_done[(gb - 1) % L::kScores], ((gb - 1) / L::kScores) & 1u, abort_flag, err, 0xA3);
          tc_fence_after_sync();
          const float f = moved ? exp2_approx(before - bound) : 1.f;
#pragma unroll 1
          for (int c = 0; c < kTi * L::kOTile; c += 16) {
            float o[16];
            tmem_ld_x16(o_tmem + lane_off + c, o);
            tmem_wait_ld_regs16(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= f;
            tmem_st_x16(o_tmem + lane_off + c, o);
          }
        }
        if (bound != l_bound) {
          const float f = l_bound == kPgNoBound ? 0.f : exp2_approx(l_bound - bound);
          l0 = l_bound == kPgNoBound && l0 == l0 ? 0.f : l0 * f;
          l_bound = bound;
        }
        // weights, as bf16 in the place of the scores
        if (used) {
          const uint64_t neg2 = pack_f32x2(-bound, -bound);
          uint64_t l2[2] = {pack_f32x2(l0, 0.f), 0ull};
#pragma unroll
          for (int i = 0; i < kKeys; i += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int c = i; c < i + 32; c += 2) {
              unpack_f32x2(fma_f32x2(pack_f32x2(x[c], x[c + 1]), to_log2_2, neg2), x[c], x[c + 1]);
              x[c] = exp2_approx(x[c]);
              x[c + 1] = exp2_approx(x[c + 1]);
              l2[(c / 2) & 1] = add_f32x2(l2[(c / 2) & 1], pack_f32x2(x[c], x[c + 1]));
              const __nv_bfloat162 w = __floats2bfloat162_rn(x[c], x[c + 1]);
              pk[(c - i) / 2] = *reinterpret_cast<const uint32_t*>(&w);
            }
            tmem_st_words_x16(s_at + i / 2, pk);
          }
          float l1;
          unpack_f32x2(add_f32x2(l2[0], l2[1]), l0, l1);
          l0 += l1;
          tmem_wait_st();
        }
        tc_fence_before_sync();
        __syncwarp();
        // (a barrier for each place of scores: with one for each group a warp that is a block ahead, as the third place allows, would
        // count for one that is not done)
        if (lane == 0) mbar_arrive(&p_full[gb % L::kScores]);
      }
      gb0 += nb;
      // the part's end: the two threads' sums in units of the row's last bound
      named_bar_sync(kTcEpiBar, kPgSoft);
      if (nb > 0) paged_wait(&pv_done[(gb0 - 1) % L::kScores], ((gb0 - 1) / L::kScores) & 1u, abort_flag, err, 0xA5);
      tc_fence_after_sync();
      float bound = kPgNoBound;
      if (nb > 0) bound = bound_s[r];
      sum_s[group * N + r] = l0 != l0 ? l0 : (l_bound == kPgNoBound ? 0.f : l0 * exp2f(l_bound - bound));
      named_bar_sync(kTcEpiBar, kPgSoft);
      const float sum = sum_s[r] + sum_s[N + r];
      const PagedPart un = part_s[n & 1];
      const int way = un.way;
      const int64_t place = 2 * static_cast<int64_t>(cta) + (way == kPgHead ? 1 : 0);  // of a shared unit's part
      float f = 1.f;
      float none = 0.f;  // no number where an output is
      if (r < un.cols) {
        if (way == kPgWhole) {
          f = paged_factor(bound, sum, p.sink, p.head(un.skip + r), p.lse != nullptr && group == 0 ? p.lse + un.row0 + r : nullptr);
        } else if (group == 0) {
          __stcg(p.stats + place * 2 * N + r, bound);
          __stcg(p.stats + place * 2 * N + N + r, sum);
        }
      }
      if (used) {
        // half of the dims for each of the row's two threads, whole sectors at a time where they are aligned
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0u;
        uint16_t* out = p.out + (static_cast<int64_t>(un.row0) + r) * D;
        float* part = p.partial + (place * N + r) * D;
#pragma unroll 1
        for (int d = group * (D / 2); d < (group + 1) * (D / 2); d += 16) {
          float o[16];
          if (nb > 0) {
            tmem_ld_x16(o_tmem + lane_off + d, o);
            tmem_wait_ld_regs16(o);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = 0.f;
          }
          none = max3_nan(none, any_nan(o), 0.f);
          if (r < un.cols && way == kPgWhole) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const __nv_bfloat162 two = __floats2bfloat162_rn(o[j] * f, o[j + 1] * f);
              w[j / 2] = *reinterpret_cast<const uint32_t*>(&two);
            }
            if (wide) {
              st_32(out + d, w);
            } else {
              reinterpret_cast<uint4*>(out + d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(out + d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          } else if (r < un.cols) {
#pragma unroll
            for (int j = 0; j < 16; j += 4) __stcg(reinterpret_cast<float4*>(part + d + j), make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]));
          }
          __syncwarp();
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_empty);
        mbar_arrive(&part_empty[n & 1]);
      }
      // (behind it bounds and sums are written anew by the next part)
      if (bar_or(kTcEpiBar, kPgSoft, none != none && r < un.cols)) {
        // An infinite value of weight 0 (a score of minus infinity) in a block that every row sees: the rest of that row of outputs
        // becomes none either, as in blocks whose masks had the value found.
        sum_s[group * N + r] = none != none ? 1.f : 0.f;
        named_bar_sync(kTcEpiBar, kPgSoft);
        if (r < un.cols && sum_s[r] + sum_s[N + r] != 0.f) {
          const float nan = __int_as_float(0x7FFFFFFF);
          if (way == kPgWhole) {
            uint4* to = reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(un.row0) + r) * D + group * (D / 2));
#pragma unroll 1
            for (int d = 0; d < D / 16; ++d) to[d] = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
            if (p.lse != nullptr && group == 0) p.lse[un.row0 + r] = nan;
          } else if (group == 0) {
            __stcg(p.stats + place * 2 * N + N + r, nan);
          }
        }
        named_bar_sync(kTcEpiBar, kPgSoft);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax and output, a thread with a row of the block
    // All softmax warps take the same way: the block counts are those of a wait that succeeded for all of them, and
    // what they decide in a block is a vote over all.  So the hardware barriers, whose wait has no limit,
    // are passed by all or by none.
    const int etid = threadIdx.x - 32 * kPgFirstSoft;
    const int quarter = warp & 3;                                  // tensor-memory lane quarter
    const int gc = ((warp - kPgFirstSoft) >> 2) * 32;                         // this warp's columns [gc, gc + 32)
    constexpr int kC = 16;
    const int cb = gc + (lane >> 4) * 16;                          // this thread's [cb, cb + kC)
    const int r = quarter * 16 + (lane & 15);                      // its row of the block
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float to_log2 = p.to_log2[0];
    const uint64_t to_log2_2 = *reinterpret_cast<const uint64_t*>(p.to_log2);
    uint32_t gb = 0;
    uint64_t lsum[kC / 2];
    float x[kC];          // scores or weights of its columns
    uint32_t p_zero = 0u;  // bit i: this warp's part of P of even (odd) blocks is zero
    const auto load = [&](uint32_t at) {
      tmem_ld_half_x16(at, x);
      tmem_wait_ld_regs16(x);
    };
    for (int n = 0;; ++n) {
      paged_wait(&part_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, err, 0xA0);
      const int nb = part_s[n & 1].blocks;
      if (etid < N) neg_s[etid] = -kPgNoBound;
#pragma unroll
      for (int c = 0; c < kC / 2; ++c) lsum[c] = 0ull;
      if (bar_or(kTcEpiBar, kPgSoft, *abort_flag != 0)) break;
      if (__any_sync(0xffffffffu, part_s[n & 1].unit < 0)) break;
      const int* end = end_s + (n & 1) * kPgMaxTokens;
      bool used;  // some of this warp's columns are (of others nothing is read, written or kept)
      int skip, i_first, i_last;  // rows before the unit's first in its token; the tokens of this warp's columns
      {
        const PagedPart un = part_s[n & 1];
        used = gc < un.cols;
        skip = un.skip;
        i_first = p.by_H(gc + skip);
        i_last = p.by_H(max(min(gc + 32, un.cols) - 1, 0) + skip);
      }
      for (int b = 0; b < nb; ++b, ++gb) {
        const uint32_t slot = gb % kPgSlots;
        paged_wait(&blk_full[slot], (gb / kPgSlots) & 1u, abort_flag, err, 0xA1);
        const PagedBlock& blk = block_s[slot];
        const bool full = blk.full != 0, starts_run = __any_sync(0xffffffffu, blk.starts != 0) != 0;
        const int row = blk.row + r;
        const int i0 = max(blk.i0, i_first), i1 = min(blk.i1 - 1, i_last);
        const bool here = ((blk.pages >> (r >> p.pages.log_rows)) & 1u) != 0;
        const int tail = blk.tail;
        __syncwarp();
        if (lane == 0) mbar_arrive(&blk_empty[slot]);
        const bool some = __any_sync(0xffffffffu, used && i0 <= i1) != 0;  // some of this warp's columns are the block's
        uint32_t mask = 0xFFFFFFFFu;         // the columns that see this thread's row
        uint32_t run = 0u;                   // the columns of the block's tokens
        if (!full) {
          mask = 0u;
          // a row is seen where 0 <= end - 1 - row < span
          const unsigned span = !here ? 0u : static_cast<unsigned>(row < p.first ? INT32_MAX : p.window);
#pragma unroll 1
          for (int i = i0; i <= i1; ++i) {
            const int c = i * p.H - skip - cb;  // the token's first column
            const uint32_t bits = low_bits(min(max(c + p.H, 0), kC)) & ~low_bits(min(max(c, 0), kC));
            run |= bits;
            if (static_cast<unsigned>(end[i] - 1 - row) < span) mask |= bits;
          }
        }
        const uint32_t s_at = s_tmem + N * (gb & 1u) + lane_off + gc;
        uint8_t* p_row = p_s + (gb & 1u) * (kKeys * 128);
        paged_wait(&s_full[gb & 1u], (gb >> 1) & 1u, abort_flag, err, 0xA2);
        tc_fence_after_sync();
        if (tail < kKeys) {  // rows that may never have been written: weights of 0 times what is no number would be none
          for (int c = 0; c < kCh; ++c) {
            uint8_t* chunk = kv_s + ((gb * kTi + c / 2) % kRing) * L::kTileBytes + (c & 1) * L::kChunkBytes;
            for (int i = tail * 128 + etid * 16; i < L::kChunkBytes; i += kPgSoft * 16)
              *reinterpret_cast<uint4*>(chunk + i) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        const bool checks = !full && r < tail;  // whether scores that are no numbers matter
        // weights by the bounds as they are, 0 where a column does not see the row, written into the bf16 row P[row r]; x keeps
        // them.  True where an exponent exceeds its bound by more than 2^8, or a score is no number in a block that not every
        // column sees all of.
        if (gb >= 2) paged_wait(&pv_done[gb & 1u], ((gb >> 1) - 1) & 1u, abort_flag, err, 0xA4);  // P's place is free
        const auto weights = [&]() {
          load(s_at);
          uint64_t none = 0ull;  // is a number where every score is
          if (checks) {
#pragma unroll
            for (int c = 0; c < kC; c += 2) none = fma_f32x2(pack_f32x2(x[c], x[c + 1]), 0ull, none);
          }
          float over = -INFINITY;
#pragma unroll
          for (int c = 0; c < kC; c += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
              const float4 nm = *reinterpret_cast<const float4*>(neg_s + cb + c + i);
              float y[4];
              unpack_f32x2(fma_f32x2(pack_f32x2(x[c + i], x[c + i + 1]), to_log2_2, pack_f32x2(nm.x, nm.y)), y[0], y[1]);
              unpack_f32x2(fma_f32x2(pack_f32x2(x[c + i + 2], x[c + i + 3]), to_log2_2, pack_f32x2(nm.z, nm.w)), y[2], y[3]);
              if (!full) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (((mask >> (c + i + k)) & 1u) == 0u) y[k] = -INFINITY;
              }
              over = max3(max3(over, y[0], y[1]), y[2], y[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) x[c + i + k] = exp2_approx(y[k]);
              const __nv_bfloat162 w0 = __floats2bfloat162_rn(x[c + i], x[c + i + 1]), w1 = __floats2bfloat162_rn(x[c + i + 2], x[c + i + 3]);
              pk[i / 2] = *reinterpret_cast<const uint32_t*>(&w0);
              pk[i / 2 + 1] = *reinterpret_cast<const uint32_t*>(&w1);
            }
            *reinterpret_cast<uint4*>(p_row + swz128(r, 2 * (cb + c))) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
          float n0, n1;
          unpack_f32x2(none, n0, n1);
          return over > kTcLazyLog2 || n0 != n0 || n1 != n1;
        };
        bool raise = starts_run;
        if (some && !starts_run) raise = weights();
        if (bar_or(kTcEpiBar, kPgSoft, raise)) {
          // A run's first block, and rarely another: a bound is raised, or a masked row holds what is no number.  The largest
          // score of each column:
          const auto largest = [&]() {
            bool odd = false;  // (scores of columns of other tokens show nothing: their q may hold anything)
            load(s_at);
#pragma unroll
            for (int c = 0; c < kC; ++c) {
              odd |= checks && ((run >> c) & 1u) != 0u && !(fabsf(x[c]) < INFINITY);
              x[c] = ((mask >> c) & 1u) != 0u ? x[c] * to_log2 : -INFINITY;
            }
            xpose_reduce<kC>(x, lane, [](float v, float w) { return fmaxf(v, w); });
            atomicMax(top_s + cb + lane % kC, ordered(x[0]));
            return odd;
          };
          bool odd = false;
          if (some) odd = largest();
          if (bar_or(kTcEpiBar, kPgSoft, odd)) {
            // 0 times such a value would still be no number in the weighted sum.  So a row that holds one is taken out of the
            // products, and the columns that see it get a sum that is no number.
            bool bad = false;
            const auto at = [&](int c) { return kv_s + ((gb * kTi + c / 2) % kRing) * L::kTileBytes + (c & 1) * L::kChunkBytes + r * 128; };
#pragma unroll 1
            for (int c = 0; c < kCh; ++c) {
              const uint32_t tile = gb * kTi + c / 2;
              paged_wait(&kv_full[tile % kRing], (tile / kRing) & 1u, abort_flag, err, 0xA6);
#pragma unroll 1
              for (int i = 0; i < 8; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(at(c) + i * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) bad |= (w[k] & 0x7F80u) == 0x7F80u || (w[k] & 0x7F800000u) == 0x7F800000u;
              }
            }
            bad = bad && !full;  // (a full block's row is seen by all columns: what comes of it is theirs)
            if (etid < N) top_s[etid] = ordered(-INFINITY);
            named_bar_sync(kTcEpiBar, kPgSoft);
            if (bad) {
              if (cb == 0)
#pragma unroll 1
                for (int c = 0; c < kCh; ++c)
#pragma unroll 1
                  for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(at(c) + i * 16) = make_uint4(0u, 0u, 0u, 0u);
              const float nan = __int_as_float(0x7FFFFFFF);
#pragma unroll
              for (int c = 0; c < kC; c += 2) {
                float s0, s1;
                unpack_f32x2(lsum[c / 2], s0, s1);
                lsum[c / 2] = pack_f32x2(((mask >> c) & 1u) != 0u ? nan : s0, ((mask >> c) & 2u) != 0u ? nan : s1);
              }
              mask = 0u;
            }
            if (some) largest();
            named_bar_sync(kTcEpiBar, kPgSoft);
          }
          bool moved = false;
          if (etid < N) {
            const float bm = from_ordered(top_s[etid]), mo = -neg_s[etid];
            const float mn = bm > mo + kTcLazyLog2 ? bm : mo;
            moved = mn != mo && mo != kPgNoBound;
            alpha_s[etid] = moved ? exp2f(mo - mn) : 1.f;
            neg_s[etid] = -mn;
            top_s[etid] = ordered(-INFINITY);
          }
          moved = bar_or(kTcEpiBar, kPgSoft, moved);
          if (moved && b > 0) {
            // sums and output accumulators of earlier blocks follow (the weighted sum of the block two before the last was waited for, so
            // the phase is the barrier's next)
            paged_wait(&pv_done[(gb - 1) % L::kScores], ((gb - 1) / L::kScores) & 1u, abort_flag, err, 0xA3);
            tc_fence_after_sync();
            if (used) {
#pragma unroll
              for (int c = 0; c < kC; c += 2)
                lsum[c / 2] = fma_f32x2(lsum[c / 2], pack_f32x2(alpha_s[cb + c], alpha_s[cb + c + 1]), 0ull);
#pragma unroll 1
              for (int m = 0; m < 2 * kTi; ++m) {  // (this thread: its dim of every tile, its warp's columns)
                const int c0 = gc + (m & 1) * 16;
                tmem_ld_x16(o_tmem + lane_off + N * (m >> 1) + c0, x);
                tmem_wait_ld_regs16(x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= alpha_s[c0 + j];
                tmem_st_x16(o_tmem + lane_off + N * (m >> 1) + c0, x);
              }
              tmem_wait_st();
            }
          }
          if (some) weights();
        }
        if (some) {
          p_zero &= ~(1u << (gb & 1u));
        } else if (used && ((p_zero >> (gb & 1u)) & 1u) == 0u) {
          p_zero |= 1u << (gb & 1u);
#pragma unroll
          for (int c = 0; c < kC; c += 8) *reinterpret_cast<uint4*>(p_row + swz128(r, 2 * (cb + c))) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_shared();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[gb % L::kScores]);
        if (some) {
#pragma unroll
          for (int c = 0; c < kC; c += 2) lsum[c / 2] = add_f32x2(lsum[c / 2], pack_f32x2(x[c], x[c + 1]));
        }
      }
      // the part's end: sums over the block's rows (P's place holds the quarters' once it is free)
      if (nb > 0) paged_wait(&pv_done[(gb - 1) % L::kScores], ((gb - 1) / L::kScores) & 1u, abort_flag, err, 0xA5);
      tc_fence_after_sync();
      named_bar_sync(kTcEpiBar, kPgSoft);
      float* red_s = reinterpret_cast<float*>(p_s);  // [4][N]
      p_zero = 0u;
#pragma unroll
      for (int c = 0; c < kC; c += 2) unpack_f32x2(lsum[c / 2], x[c], x[c + 1]);
      xpose_reduce<kC>(x, lane, [](float v, float w) { return v + w; });
      red_s[quarter * N + cb + lane % kC] = x[0];
      named_bar_sync(kTcEpiBar, kPgSoft);
      const PagedPart un = part_s[n & 1];  // (its place is held until the end of the part)
      const int way = un.way;
      const int64_t place = 2 * static_cast<int64_t>(cta) + (way == kPgHead ? 1 : 0);  // of a shared unit's part
      if (etid < un.cols) {
        const float l = (red_s[etid] + red_s[N + etid]) + (red_s[2 * N + etid] + red_s[3 * N + etid]);
        if (way == kPgWhole) {
          alpha_s[etid] = paged_factor(-neg_s[etid], l, p.sink, p.head(un.skip + etid), p.lse != nullptr ? p.lse + un.row0 + etid : nullptr);
        } else {
          __stcg(p.stats + place * 2 * N + etid, -neg_s[etid]);
          __stcg(p.stats + place * 2 * N + N + etid, l);
        }
      }
      named_bar_sync(kTcEpiBar, kPgSoft);
      const int dim = quarter * 32 + lane;           // of a tile
      uint32_t none = 0u;                            // this warp's columns with an output that is no number
      if (used) {
#pragma unroll 1
        for (int m = 0; m < kTi; ++m) {
#pragma unroll 1
          for (int c = gc; c < gc + 32; c += 16) {
            float o[16];
            if (nb > 0) {
              tmem_ld_x16(o_tmem + lane_off + N * m + c, o);
              tmem_wait_ld_regs16(o);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = 0.f;
            }
            const float odd = any_nan(o);
            if (__any_sync(0xffffffffu, odd != odd)) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (o[j] != o[j]) none |= 1u << (c - gc + j);
            }
            if (way != kPgWhole) {
              float* to = p.partial + (place * N + c) * D + 128 * m + dim;
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (c + j < un.cols) __stcg(to + j * D, o[j]);
              continue;
            }
            // Neighbouring lanes (dims) trade halves of a pair of columns, so that each stores two dims of one: 64
            // contiguous bytes per column and warp.
            const bool second = (lane & 1) != 0;
            uint16_t* dst = p.out + (static_cast<int64_t>(un.row0) + c + (second ? 1 : 0)) * D + 128 * m + (dim & ~1);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 f = *reinterpret_cast<const float2*>(alpha_s + c + j);
              const __nv_bfloat162 two = __floats2bfloat162_rn(o[j] * f.x, o[j + 1] * f.y);
              const uint32_t w = *reinterpret_cast<const uint32_t*>(&two);
              const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 1);
              const uint32_t own = second ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
              if (c + j + (second ? 1 : 0) < un.cols) *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(j) * D) = own;
            }
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_empty);
        mbar_arrive(&part_empty[n & 1]);
      }
      none &= low_bits(max(un.cols - gc, 0));
      // (behind it alpha_s, neg_s and P's place are written anew by the next part)
      if (bar_or(kTcEpiBar, kPgSoft, none != 0u)) {
        // As at D <= 256: the rest of a row of outputs with one that is no number becomes none either.
        none = __reduce_or_sync(0xffffffffu, none);
        red_s[quarter * N + gc + lane] = ((none >> lane) & 1u) != 0u ? 1.f : 0.f;
        named_bar_sync(kTcEpiBar, kPgSoft);
        const float nan = __int_as_float(0x7FFFFFFF);
#pragma unroll 1
        for (int c = gc; c < min(gc + 32, un.cols); ++c) {
          if (red_s[c] + red_s[N + c] + red_s[2 * N + c] + red_s[3 * N + c] == 0.f) continue;
          if (way == kPgWhole) {
            for (int m = 0; m < kTi; ++m) p.out[(static_cast<int64_t>(un.row0) + c) * D + 128 * m + dim] = 0x7FFFu;
            if (p.lse != nullptr && quarter == 0 && lane == 0) p.lse[un.row0 + c] = nan;
          } else if (quarter == 0 && lane == 0) {
            __stcg(p.stats + place * 2 * N + N + c, nan);
          }
        }
        named_bar_sync(kTcEpiBar, kPgSoft);
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (*abort_flag != 0 && warp == kPgFirstLoad) {
    // Some role gave up, perhaps after the loading warps were done: copies that nobody waited for land before the CTA ends.
    const uint32_t nq = issued_s[L::kLoaders];
    for (uint32_t i = nq > kQb ? nq - kQb : 0; i < nq; ++i) mbar_wait_drain(&q_full[i % kQb], (i / kQb) & 1u);
    tiles_in_flight<kRing, L::kLoaders>(issued_s, [&](uint32_t place, uint32_t parity) { mbar_wait_drain(&kv_full[place], parity); });
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the join may be made ready: it waits for this grid's end)
  if (warp == 0) tmem_dealloc(tbase, 512);
}

// ------------------------------------------------------------------------------------ shared units

constexpr int kPgJoinThreads = 128;  // (eight blocks an SM, as the launch counts on: with registers for seven drafts took 4 us more)
constexpr int kPgJoinWarps = kPgJoinThreads / 32;
constexpr int kPgMaxCtas = 512;    // CTAs that may share a unit
// Up to so many parts a warp joins by itself (always: one token, of some 120 parts, 28 us; never: 22.2, but drafts 82; so: 22.5, 65).
constexpr int kPgFewParts = 8;

// Joins the parts of the units that several CTAs shared: block (i, j) an equal share j of the i-th entry's columns and pieces of
// 128 dims.  A warp takes one such item, four dims a lane (two at D = 64); where the parts are many, a block does, a quarter of
// them a warp.  The loads of eight parts are in flight at a time.
template <int D>
__global__ void __launch_bounds__(kPgJoinThreads, 8) paged_join_kernel(const PagedAttnParams p) {
  constexpr int N = paged_cols(D);
  constexpr int kPieces = D >= 128 ? D / 128 : 1;
  constexpr int kEach = D >= 128 ? 4 : 2;  // dims of a lane
  __shared__ float acc_s[kPgJoinWarps][32 * kEach];
  __shared__ float stat_s[kPgJoinWarps][2];
  wait_stream();
  const int4 e = __ldcg(p.shared + blockIdx.x);
  const int parts = min(e.z, kPgMaxCtas);
  if (parts <= 0) return;
  const int row0 = e.x, cols = e.w;  // of the unit
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // part k of the unit: the end of the first CTA's piece, the beginnings of the others'
  const auto place = [&](int k) { return 2 * (static_cast<int64_t>(e.y) + k) + (k == 0 ? 1 : 0); };
  const bool few = parts <= kPgFewParts;
  const int k0 = few ? 0 : parts * warp / kPgJoinWarps, k1 = few ? parts : parts * (warp + 1) / kPgJoinWarps;
  const int items = cols * kPieces, step = static_cast<int>(gridDim.y) * (few ? kPgJoinWarps : 1);
  for (int item = static_cast<int>(blockIdx.y) * (few ? kPgJoinWarps : 1) + (few ? warp : 0); item < items; item += step) {
    const int c = item / kPieces, d = (item % kPieces) * 128 + lane * kEach;
    float top = kPgNoBound, sum = 0.f;
    float acc[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) acc[i] = 0.f;
    constexpr int kAhead = 8;
    for (int kb = k0; kb < k1; kb += kAhead) {
      float v[kAhead][kEach];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (kb + k < k1) {
          const float* from = p.partial + (place(kb + k) * N + c) * D + d;
          if constexpr (kEach == 4) {
            const float4 w = __ldcg(reinterpret_cast<const float4*>(from));
            v[k][0] = w.x, v[k][1] = w.y, v[k][2] = w.z, v[k][3] = w.w;
          } else {
            const float2 w = __ldcg(reinterpret_cast<const float2*>(from));
            v[k][0] = w.x, v[k][1] = w.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < kEach; ++i) v[k][i] = 0.f;
        }
      }
      // lanes 0 to 7: bounds and sums of these parts
      float m = kPgNoBound, l = 0.f;
      if (lane < kAhead && kb + lane < k1) {
        m = __ldcg(p.stats + place(kb + lane) * 2 * N + c);
        l = __ldcg(p.stats + place(kb + lane) * 2 * N + N + c);
      }
      float most = m;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      most = fmaxf(top, __shfl_sync(0xffffffffu, most, 0));
      const float back = top == kPgNoBound ? 0.f : exp2f(top - most);
      top = most;
      const float f = m == kPgNoBound ? 0.f : exp2f(m - top);
      float s = l != l ? l : l * f;  // (a sum that is no number stays one, whatever its part weighs)
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      sum = (sum != sum ? sum : sum * back) + __shfl_sync(0xffffffffu, s, 0);
#pragma unroll
      for (int i = 0; i < kEach; ++i) acc[i] *= back;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float w = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
        for (int i = 0; i < kEach; ++i) acc[i] = fmaf(v[k][i], w, acc[i]);
      }
    }
    if (!few) {  // (the whole block is here)
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kEach; ++i) acc_s[warp][lane * kEach + i] = acc[i];
      if (lane == 0) {
        stat_s[warp][0] = top;
        stat_s[warp][1] = sum;
      }
      __syncthreads();
      if (warp != 0) continue;
      float most = kPgNoBound;
#pragma unroll
      for (int w = 0; w < kPgJoinWarps; ++w) most = fmaxf(most, stat_s[w][0]);
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kEach; ++i) acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kPgJoinWarps; ++w) {
        const float m = stat_s[w][0], l = stat_s[w][1];
        const float f = m == kPgNoBound ? 0.f : exp2f(m - most);
        sum += l != l ? l : l * f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) acc[i] = fmaf(acc_s[w][lane * kEach + i], f, acc[i]);
      }
      top = most;
    }
    const float f = paged_factor(top, sum, p.sink, p.head(row0 + c), p.lse != nullptr && item % kPieces == 0 && lane == 0 ? p.lse + row0 + c : nullptr);
    uint16_t* out = p.out + (static_cast<int64_t>(row0) + c) * D + d;
#pragma unroll
    for (int i = 0; i < kEach; i += 2) {
      const __nv_bfloat162 two = __floats2bfloat162_rn(acc[i] * f, acc[i + 1] * f);
      *reinterpret_cast<uint32_t*>(out + i) = *reinterpret_cast<const uint32_t*>(&two);
    }
  }
}

}  // namespace dsa
