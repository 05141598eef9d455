// Attention of each token over the rows of its sequence in a bf16 paged cache, on the tensor cores.  Token t at
// position p of sequence r sees the rows j <= p, of which with a window W only j > p - W, and j < F.  For head h
//     x_j = scale * q[t,h,:] . kv_j,   out[t,h,:] = sum_j e^{x_j} kv_j / ( sum_j e^{x_j} + e^{sink[h]} )
// (a kv row is both key and value).  Products run on bf16 operands with fp32 accumulators; the weights enter the second
// one as bf16 (off by half a step, 2^-8 of each, at most), the denominator sums them in fp32.
//
// Rows of q are (token, head) pairs, which lie one after the other; a unit is up to N of them: some consecutive
// tokens with all their heads, or N heads of one token.  The tokens of a unit need not share a sequence: the unit's
// blocks are those of its runs of tokens of one sequence, one run after the other, and a run's blocks are masked for
// the other tokens.  (A product of N = 128 columns takes 64 cycles and one of 64 takes 52 to 63, so the idle columns
// of such a block cost nothing that a unit of its own would not.)
//
// All blocks of all units, and for each unit a constant for its q and output, lie on one line that is cut into as
// many equal pieces as there are CTAs; each CTA finds its piece by a scan over the units.  So one long sequence
// uses all SMs, a batch of uneven ones keeps them equally busy, and a prompt's units go out whole but for one at
// each cut.  The parts of a unit that several CTAs share go to the workspace and are joined by a second kernel.
//
// One CTA per SM, 640 threads, per block of 128 rows:
//   scout    (warp 2)      the unit's runs and blocks; the pages of the next blocks, four blocks at a time;
//   load     (warp 1)      the rows by TMA, as D / 64 chunks of [128 rows x 128 bytes], 128-byte swizzled, page by
//                          page (a page without a row that some token sees becomes zeros: its memory is not read);
//   score    (warp 0)      S^T = KV . Q^T: M = 128 rows, N columns, K = D (tcgen05.mma kind::f16, bf16);
//   softmax  (warps 4-19)  thread = (row, N / 4 columns): weights as bf16 rows P[row][column]; the running bound of a
//                          column moves only when exceeded by more than 2^8;
//   weighted (warp 0)      O^T += KV^T . P^T: M = 128 dims (D / 128 tiles), N columns, K = 128 rows.
// Where two blocks fit (D <= 256) the score product of the next block is issued before the weighted sum of the last.
#pragma once

#include <cuda_bf16.h>

#include "attn_kv4_kernel.cuh"
#include "paged.cuh"

namespace dsa {

constexpr int kPgKeys = 128;              // rows of a block
constexpr int kPgSoftWarps = 16;
constexpr int kPgSoftThreads = 32 * kPgSoftWarps;
constexpr int kPgThreads = 128 + kPgSoftThreads;
constexpr int kPgSlots = 8;               // blocks whose pages are looked up ahead
constexpr int kPgBatch = 4;               // blocks looked up at a time
constexpr int kPgMaxTokens = 32;          // tokens of a unit: a lane of the scout each
constexpr int kPgUnitCost = 2;            // what a unit costs beside its blocks, in blocks
constexpr int kPgMinBlocks = 2;           // least piece of the line (in blocks): joining a part takes about as long
constexpr float kPgNoBound = -3e38f;      // bound of a column without rows so far

// Columns of a unit at head dimension D: with 128 the output accumulators of D = 512 would take all tensor memory.
__host__ __device__ constexpr int paged_cols(int D) { return D == 512 ? 64 : 128; }

// What the load and softmax warps know of a block.
struct PagedBlock {
  int row;         // its first row in the sequence
  int c0, c1;      // columns that it is for
  int full;        // every column sees every row
  uint32_t pages;  // bit i: page i of the block is there
  int id[8];       // pages of the block
  int pad[3];
};

// What the CTA does of a unit.
struct PagedPart {
  int unit;
  int blocks;   // of this CTA
  int way;      // kPgWhole: the CTA has all blocks; kPgHead: the first ones; kPgTail: later ones
  int pad;
};
constexpr int kPgWhole = 0, kPgHead = 1, kPgTail = 2;

template <int D>
struct PagedLayout {
  static constexpr int kCols = paged_cols(D);
  static constexpr int kStages = D <= 128 ? 4 : (D <= 256 ? 2 : 1);  // blocks held
  static constexpr int kScores = kStages < 2 ? 1 : 2;                // score accumulators
  static constexpr int kChunks = D / 64;
  static constexpr int kTiles = D >= 128 ? D / 128 : 1;              // output tiles (D = 64: half of one is zero)
  static constexpr int kChunkBytes = kPgKeys * 128;
  static constexpr int kStageBytes = 2 * kTiles * kChunkBytes;
  static constexpr int kTileBytes = (D >= 128 ? 2 : 1) * kChunkBytes;  // of a tile that are loaded
  static constexpr int kQChunkBytes = kCols * 128;
  static constexpr int kKv = 0;
  static constexpr int kQ = kKv + kStages * kStageBytes;
  static constexpr int kP = kQ + kChunks * kQChunkBytes;          // bf16, kCols / 64 chunks of [128 rows][64 columns]
  static constexpr int kMax = kP + kPgKeys * kCols * 2;           // float [cols] running bounds (log2 units)
  static constexpr int kAlpha = kMax + kCols * 4;                 // float [cols] rescale / output factors, or reduced bounds
  static constexpr int kEnd = kAlpha + kCols * 4;                 // int [2][cols] by unit: rows below this are seen
  static constexpr int kBlocks = kEnd + 2 * kCols * 4;            // PagedBlock [slots]
  static constexpr int kParts = kBlocks + kPgSlots * static_cast<int>(sizeof(PagedBlock));  // PagedPart [2]
  static constexpr int kPlan = kParts + 2 * static_cast<int>(sizeof(PagedPart));            // int [12]
  static constexpr int kBar = kPlan + 48;
  static constexpr int kNumBars = 14 + 2 * kPgSlots + 2 * kStages * kTiles;
  static constexpr int kSmem = kBar + kNumBars * 8;
  // tensor memory: S^T (kScores of them) from column 0, O^T tile m from column kCols (kScores + m)
};
static_assert(sizeof(PagedBlock) == 64 && sizeof(PagedPart) == 16, "layout");

// ------------------------------------------------------------------------------------ units and runs

struct PagedUnit {
  int t0, n;    // tokens
  int h0;       // first head
  int cols;     // columns in use
};

__device__ __forceinline__ PagedUnit paged_unit(const PagedAttnParams& p, int u, int N) {
  PagedUnit r;
  if (p.groups > 1) {
    r.t0 = u / p.groups;
    r.n = 1;
    r.h0 = (u % p.groups) * N;
    r.cols = min(N, p.H - r.h0);
  } else {
    r.t0 = u * p.tokens;
    r.n = min(p.tokens, p.T - r.t0);
    r.h0 = 0;
    r.cols = r.n * p.H;
  }
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
  int low, high, some;  // union
  int all_low, all_end;  // what every token sees: [all_low, all_end)
  __device__ __forceinline__ void start() {
    low = INT32_MAX;
    high = some = all_low = 0;
    all_end = INT32_MAX;
  }
  __device__ __forceinline__ void add(const PagedAttnParams& p, int end) {
    const int lo = max(0, end - p.window);
    low = min(low, lo);
    all_low = max(all_low, lo);
    high = max(high, end);
    all_end = min(all_end, end);
    some = max(some, min(p.first, end));
  }
  // blocks [0, a) and [b, b + the rest); the number of them
  __device__ __forceinline__ int blocks(const PagedAttnParams& p, int& a, int& b) const {
    const int rows = min(high, p.pages.M << p.pages.log_rows);
    const auto up_to = [](int n) { return n > 0 ? (n - 1) / kPgKeys + 1 : 0; };
    b = low / kPgKeys;
    a = min(up_to(min(some, rows)), b);
    return a + max(0, up_to(rows) - b);
  }
};

// Blocks of a unit.
__device__ __forceinline__ int paged_blocks(const PagedAttnParams& p, const PagedUnit& u) {
  int n = 0, seq = -1, a, b;
  PagedRun run;
  run.start();
  for (int i = 0; i <= u.n; ++i) {
    int s = -1, end = 0;
    if (i < u.n) paged_token(p, u.t0 + i, s, end);
    if (s != seq || i == u.n) {
      if (seq >= 0) n += run.blocks(p, a, b);
      run.start();
      seq = s;
    }
    if (s >= 0) run.add(p, end);
  }
  return n;
}

// Factor of a column's outputs whose weights' bound is m (log2 units) and whose denominator is l, in units of 2^m,
// without the sink; writes the natural log of the whole denominator where lse is given (a NaN stays one).
__device__ __forceinline__ float paged_factor(float m, float l, const float* sink, int h, float* lse) {
  if (l != l) {
    if (lse != nullptr) *lse = l;
    return l;
  }
  return softmax_factor(m, l, sink, h, lse);
}

// An fp32 value as an int of the same order (no NaN).
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_ordered(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7FFFFFFF)); }

template <int D>
__global__ void __launch_bounds__(kPgThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap qmap,
                      const PagedAttnParams p, int min_blocks, unsigned* err) {
  using L = PagedLayout<D>;
  constexpr int N = L::kCols;
  constexpr int kCh = L::kChunks;
  constexpr int kTi = L::kTiles;
  constexpr int kSt = L::kStages;
  constexpr int kSc = L::kScores;
  constexpr int kC = N / 4;  // columns of a softmax thread
  extern __shared__ __align__(1024) uint8_t paged_smem[];
  uint8_t* smem = paged_smem;
  uint8_t* kv_s = smem + L::kKv;
  uint8_t* q_s = smem + L::kQ;
  uint8_t* p_s = smem + L::kP;
  float* max_s = reinterpret_cast<float*>(smem + L::kMax);
  float* alpha_s = reinterpret_cast<float*>(smem + L::kAlpha);
  int* end_s = reinterpret_cast<int*>(smem + L::kEnd);
  PagedBlock* block_s = reinterpret_cast<PagedBlock*>(smem + L::kBlocks);
  PagedPart* part_s = reinterpret_cast<PagedPart*>(smem + L::kParts);
  volatile int* plan_s = reinterpret_cast<volatile int*>(smem + L::kPlan);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* p_full = bars + 2;
  uint64_t* pv_done = bars + 3;
  uint64_t* o_empty = bars + 4;
  uint64_t* drain = bars + 5;
  uint64_t* part_full = bars + 6;   // [2]
  uint64_t* part_empty = bars + 8;  // [2]
  uint64_t* s_full = bars + 10;     // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 12);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* blk_full = bars + 14;   // [slots]
  uint64_t* blk_empty = blk_full + kPgSlots;
  uint64_t* kv_full = blk_empty + kPgSlots;  // [stage][tile]
  uint64_t* kv_empty = kv_full + kSt * kTi;

  if ((smem_addr(smem) & 1023u) != 0u) {  // (the swizzle goes by addresses; nothing else lies before this memory)
    if (threadIdx.x == 0) record_error(err, kErrPlan);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if constexpr (D == 64) {  // the upper half of a 64-dim row's tile stays zero
    for (int s = 0; s < kSt; ++s)
      for (int i = threadIdx.x; i < L::kChunkBytes / 16; i += kPgThreads)
        reinterpret_cast<uint4*>(kv_s + s * L::kStageBytes + L::kChunkBytes)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (threadIdx.x < kPgSlots * sizeof(PagedBlock) / 4) reinterpret_cast<int*>(block_s)[threadIdx.x] = 0;
  if (threadIdx.x < 2 * sizeof(PagedPart) / 4) reinterpret_cast<int*>(part_s)[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(p_full, kPgSoftWarps);
    mbar_init(pv_done, 1);
    mbar_init(o_empty, kPgSoftWarps);
    mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&part_full[i], 1);
      mbar_init(&part_empty[i], 2 + kPgSoftWarps);
      mbar_init(&s_full[i], 1);
    }
    for (int i = 0; i < kPgSlots; ++i) {
      mbar_init(&blk_full[i], 1);
      mbar_init(&blk_empty[i], 1 + kPgSoftWarps);
    }
    for (int i = 0; i < kSt * kTi; ++i) {
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
  // Cost of a unit: its blocks and kPgUnitCost.  [from, to) of the line is this CTA's.  A unit belongs to the CTA on
  // whose piece it starts (that one has at least one of its blocks) and to those whose pieces its blocks reach into.
  int64_t* scan = reinterpret_cast<int64_t*>(p_s);  // [threads + 1] (P's place; 640 * 8 bytes)
  const int u_first = static_cast<int>(static_cast<int64_t>(p.units) * threadIdx.x / kPgThreads);
  const int u_last = static_cast<int>(static_cast<int64_t>(p.units) * (threadIdx.x + 1) / kPgThreads);
  int64_t mine = 0;
  for (int u = u_first; u < u_last; ++u) mine += paged_blocks(p, paged_unit(p, u, N)) + kPgUnitCost;
  scan[threadIdx.x] = mine;
  __syncthreads();
  if (warp == 0) {
    int64_t base = 0;
    for (int i = 0; i < kPgThreads; i += 32) {
      const int64_t v = scan[i + lane];
      int64_t s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t other = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += other;
      }
      scan[i + lane] = base + s - v;  // before thread i + lane's units
      base += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) scan[kPgThreads] = base;
  }
  __syncthreads();
  const int64_t line = scan[kPgThreads];
  const int64_t ctas = max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), line / min_blocks));
  const int cta = static_cast<int>(blockIdx.x);
  const int64_t from = cta < ctas ? line * cta / ctas : line, to = cta < ctas ? line * (cta + 1) / ctas : line;
  if (u_first < u_last) {
    int64_t at = scan[threadIdx.x];
    const int64_t end = at + mine;
    // the thread whose units the piece starts (ends) on walks over them again
    const bool has_from = from < to && at <= from && from < end, has_to = from < to && at < to && to <= end;
    if (has_from || has_to) {
      for (int u = u_first; u < u_last; ++u) {
        const int nb = paged_blocks(p, paged_unit(p, u, N));
        const int64_t next = at + nb + kPgUnitCost;
        if (at <= from && from < next) {
          plan_s[0] = u;
          plan_s[1] = static_cast<int>(min(from - at, static_cast<int64_t>(nb)));  // its first block here
          plan_s[4] = from == at;                                                    // it starts here
        }
        if (at < to && to <= next) {
          plan_s[2] = u;
          plan_s[3] = static_cast<int>(min(to - at, static_cast<int64_t>(nb)));  // the end of its blocks here
          // the last CTA that has one of its blocks: the one on whose piece the last of them lies
          plan_s[5] = static_cast<int>(((at + max(nb, 1)) * ctas - 1) / line);
          plan_s[6] = nb;
        }
        at = next;
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tbase = *tmem_slot;
  const uint32_t s_tmem = tbase;
  const uint32_t o_tmem = tbase + N * kSc;
  const bool idle = from >= to;
  const int unit0 = idle ? 0 : plan_s[0], unit1 = idle ? -1 : plan_s[2];
  const int from_block = plan_s[1], to_block = plan_s[3];
  const bool starts = plan_s[4] != 0;
  const int last_cta = plan_s[5], last_blocks = plan_s[6];
  // [units <= CTAs] by unit (written by the CTA that it starts on), else by CTA
  const bool by_unit = p.units <= static_cast<int>(gridDim.x);
  if (threadIdx.x == 0) {
    if (!by_unit) {
      const bool shared = !idle && to_block < last_blocks && (unit1 > unit0 || starts);
      p.shared[cta] = shared ? make_int4(unit1, cta, last_cta - cta + 1, 0) : make_int4(0, 0, 0, 0);
    } else if (!idle) {
      for (int u = starts ? unit0 : unit0 + 1; u <= unit1; ++u)
        p.shared[u] = u == unit1 && to_block < last_blocks ? make_int4(u, cta, last_cta - cta + 1, 0) : make_int4(0, 0, 0, 0);
    }
  }
  // the unit's first block here, the end of its blocks here and what this CTA does of it (nb: all its blocks)
  const auto part_of = [&](int u, int nb, int& b0, int& b1) -> int {
    b0 = u == unit0 ? from_block : 0;
    b1 = u == unit1 ? to_block : nb;
    if (u == unit0 && !starts) return kPgTail;
    return b1 < nb ? kPgHead : kPgWhole;
  };
  const auto gone = [&]() -> bool { return __any_sync(0xffffffffu, *abort_flag != 0) != 0; };

  if (warp == 2) {
    // ------------------------------------------------------------------ scout
    uint32_t gb = 0;  // blocks of this CTA so far
    int n = 0;        // parts of this CTA so far
    for (int u = unit0; u <= unit1; ++u) {
      if (gone()) break;
      const PagedUnit un = paged_unit(p, u, N);
      int seq = -1, end = 0;
      if (lane < un.n) paged_token(p, un.t0 + lane, seq, end);
      const int nb = paged_blocks(p, un);
      int b0, b1;
      const int way = part_of(u, nb, b0, b1);
      if (way == kPgTail && b0 >= b1) continue;  // (its blocks end before this CTA's piece)
      if (n > 1) mbar_wait(&part_empty[n & 1], static_cast<uint32_t>((n >> 1) - 1) & 1u, abort_flag, err, 0x80);
      if (gone()) break;
      for (int i = 0; i < un.n; ++i) {
        const int e = __shfl_sync(0xffffffffu, end, i);
        const int c_end = p.groups > 1 ? un.cols : (i + 1) * p.H;
        for (int c = (p.groups > 1 ? 0 : i * p.H) + lane; c < c_end; c += 32) end_s[(n & 1) * N + c] = e;
      }
      for (int c = un.cols + lane; c < N; c += 32) end_s[(n & 1) * N + c] = 0;
      if (lane == 0) {
        part_s[n & 1].unit = u;
        part_s[n & 1].blocks = b1 - b0;
        part_s[n & 1].way = way;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&part_full[n & 1]);
      ++n;
      // the runs, one after the other
      int before = 0;  // blocks of the runs before
      bool ok = true;
      for (int i = 0; ok && i < un.n && before < b1;) {
        const int s = __shfl_sync(0xffffffffu, seq, i);
        const int first_token = i;
        PagedRun run;
        run.start();
        for (; i < un.n && __shfl_sync(0xffffffffu, seq, i) == s; ++i) run.add(p, __shfl_sync(0xffffffffu, end, i));
        if (s < 0) continue;
        int ra, rb;
        const int count = run.blocks(p, ra, rb);
        const bool whole = first_token == 0 && i == un.n;
        const int c0 = p.groups > 1 ? 0 : first_token * p.H, c1 = p.groups > 1 ? un.cols : i * p.H;
        const int32_t* table = p.pages.table + static_cast<int64_t>(s) * p.pages.M;
        const int k_end = min(count, b1 - before);
        for (int k0 = max(0, b0 - before); ok && k0 < k_end; k0 += kPgBatch) {
          // lane = (block of the batch, page of the block)
          const int k = min(k0 + (lane >> 3), k_end - 1);
          const int row = (k < ra ? k : rb + k - ra) * kPgKeys;
          const int at = row + ((lane & 7) << p.pages.log_rows);  // its first row (a page of more than 128: the block's)
          bool there = ((lane & 7) << p.pages.log_rows) < kPgKeys;
          // rows [at, at + box) that some token of the run sees
          there = there && (at < run.some || (at < run.high && at - run.low > -p.box_rows));
          const int index = at >> p.pages.log_rows;
          int page = -1;
          if (there && index < p.pages.M) page = ld_after_wait(table + index);
          if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.pages.P)) page = -1;
          const uint32_t mapped = __ballot_sync(0xffffffffu, page >= 0);
          const uint32_t wanted = __ballot_sync(0xffffffffu, ((lane & 7) << p.pages.log_rows) < kPgKeys);
          for (int j = 0; j < kPgBatch && k0 + j < k_end; ++j, ++gb) {
            const uint32_t slot = gb % kPgSlots;
            if (gb >= kPgSlots) mbar_wait(&blk_empty[slot], (gb / kPgSlots - 1) & 1u, abort_flag, err, 0x81);
            if (gone()) {
              ok = false;
              break;
            }
            PagedBlock& blk = block_s[slot];
            if ((lane >> 3) == j) blk.id[lane & 7] = page;
            if (lane == 8 * j) {
              const uint32_t have = (mapped >> (8 * j)) & 0xFFu, want = (wanted >> (8 * j)) & 0xFFu;
              blk.row = row;
              blk.c0 = c0;
              blk.c1 = c1;
              blk.pages = have;
              blk.full = whole && have == want && row <= run.all_end - kPgKeys &&
                         (row >= run.all_low || row <= p.first - kPgKeys);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&blk_full[slot]);
          }
        }
        before += count;
      }
      if (!ok) break;
    }
    // the end: a part without a unit
    if (!gone()) {
      if (n > 1) mbar_wait(&part_empty[n & 1], static_cast<uint32_t>((n >> 1) - 1) & 1u, abort_flag, err, 0x82);
      if (!gone() && lane == 0) {
        part_s[n & 1].unit = -1;
        part_s[n & 1].blocks = 0;
        mbar_arrive(&part_full[n & 1]);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ load
    uint32_t gb = 0, nq = 0;   // blocks and q's of this CTA so far
    uint32_t tiles = 0;        // tiles whose copies were issued
    int pages = kPgKeys >> p.pages.log_rows;
    if (pages == 0) pages = 1;
    const int rows = 1 << p.pages.log_rows;
    const int none = max(1, p.pages.P << p.pages.log_rows);  // a row behind the last page: the copy fills in zeros
    for (int n = 0;; ++n) {
      mbar_wait(&part_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, err, 0x83);
      if (gone()) break;
      const int u = part_s[n & 1].unit;
      const int nb = part_s[n & 1].blocks;
      __syncwarp();
      if (lane == 0) mbar_arrive(&part_empty[n & 1]);
      if (u < 0) break;
      if (nb == 0) continue;
      const PagedUnit un = paged_unit(p, u, N);
      // q's place is free once the score products of the part before are done
      if (nq > 0) mbar_wait(q_empty, (nq - 1) & 1u, abort_flag, err, 0x84);
      if (gone()) break;
      ++nq;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, kCh * L::kQChunkBytes);
        const int y = un.t0 * p.H + un.h0;
        for (int c = 0; c < kCh; ++c) tma_load_2d(q_s + c * L::kQChunkBytes, &qmap, q_full, 64 * c, y);
      }
      __syncwarp();
      bool ok = true;
      for (int b = 0; b < nb; ++b, ++gb) {
        const uint32_t slot = gb % kPgSlots;
        const int st = static_cast<int>(gb % kSt);
        mbar_wait(&blk_full[slot], (gb / kPgSlots) & 1u, abort_flag, err, 0x85);
        if (gone()) {
          ok = false;
          break;
        }
        const PagedBlock& blk = block_s[slot];
        const int i = lane >> 1;  // page of the block
        int y = none;
        if (i < pages && blk.id[i & 7] >= 0) y = (blk.id[i & 7] << p.pages.log_rows) + (blk.row & (rows - 1));
        __syncwarp();
        if (lane == 0) mbar_arrive(&blk_empty[slot]);
#pragma unroll
        for (int m = 0; m < kTi; ++m) {
          if (gb >= kSt) mbar_wait(&kv_empty[st * kTi + m], (gb / kSt - 1) & 1u, abort_flag, err, 0x86);
          if (gone()) {
            ok = false;
            break;
          }
          ++tiles;
          if (lane == 0) mbar_arrive_expect_tx(&kv_full[st * kTi + m], L::kTileBytes);
          __syncwarp();
          const int c = 2 * m + (lane & 1);
          if (i < pages && c < kCh)
            tma_load_2d(kv_s + st * L::kStageBytes + c * L::kChunkBytes + i * p.box_rows * 128, &kvmap, &kv_full[st * kTi + m], 64 * c, y);
        }
        if (!ok) break;
      }
      if (!ok) break;
    }
    if (gone()) {  // copies in flight land before the CTA ends
      if (nq > 0) mbar_wait_drain(q_full, (nq - 1) & 1u);
      for (uint32_t i = tiles > kSt * kTi ? tiles - kSt * kTi : 0; i < tiles; ++i)
        mbar_wait_drain(&kv_full[(i / kTi) % kSt * kTi + i % kTi], (i / (kSt * kTi)) & 1u);
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------------ MMA issuer (the whole warp, one thread elected)
    const uint32_t on = elect_one();
    const auto wait = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, site)) != 0;
    };
    constexpr uint32_t id_qk = idesc_bf16(kPgKeys, N, false, false);
    constexpr uint32_t id_pv = idesc_bf16(128, N, true, true);
    const uint64_t kv_k = desc_sw128(smem_addr(kv_s), 16, 1024);                // K-major: rows x dims
    const uint64_t q_k = desc_sw128(smem_addr(q_s), 16, 1024);                  // K-major: columns x dims
    const uint64_t kv_mn = desc_sw128(smem_addr(kv_s), L::kChunkBytes, 1024);   // MN-major: dims x rows
    const uint64_t p_mn = desc_sw128(smem_addr(p_s), kPgKeys * 128, 1024);      // MN-major: columns x rows
    const auto score = [&](uint32_t gb) -> bool {
      const uint32_t st = gb % kSt;
      const uint64_t a = kv_k + st * (L::kStageBytes >> 4);
#pragma unroll
      for (int c = 0; c < kCh; ++c) {
        if ((c & 1) == 0) {
          if (!wait(&kv_full[st * kTi + c / 2], (gb / kSt) & 1u, 0x90)) return false;
          tc_fence_after_sync();
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t ad = a + ((c * L::kChunkBytes + kk * 32) >> 4), bd = q_k + ((c * L::kQChunkBytes + kk * 32) >> 4);
          if (c == 0 && kk == 0)
            mma_f16_if<false>(on, s_tmem + N * (gb % kSc), ad, bd, id_qk, 0u);
          else
            mma_f16_if<true>(on, s_tmem + N * (gb % kSc), ad, bd, id_qk);
        }
      }
      mma_commit_if(on, &s_full[gb % kSc]);
      return true;
    };
    uint32_t gb = 0;
    uint32_t nq = 0, no = 0;  // parts with blocks so far, parts so far
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!wait(&part_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, 0x91)) break;
      const int u = __shfl_sync(0xffffffffu, part_s[n & 1].unit, 0);
      const int nb = __shfl_sync(0xffffffffu, part_s[n & 1].blocks, 0);
      if (lane == 0) mbar_arrive(&part_empty[n & 1]);
      __syncwarp();
      if (u < 0) break;
      ++no;
      if (nb == 0) continue;
      if (!wait(q_full, nq & 1u, 0x92)) break;
      ++nq;
      if (!score(gb)) break;
      if (nb == 1) mma_commit_if(on, q_empty);  // (after the part's last score product)
      for (int b = 0; b < nb; ++b, ++gb) {
        if (kSt > 1 && b + 1 < nb) {
          if (!score(gb + 1)) {
            ok = false;
            break;
          }
          if (b + 2 == nb) mma_commit_if(on, q_empty);
        }
        if (!wait(p_full, gb & 1u, 0x93)) {
          ok = false;
          break;
        }
        // the part's first weighted sum overwrites O: the previous part's output must be read
        if (b == 0 && no > 1 && !wait(o_empty, (no - 2) & 1u, 0x94)) {
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
          for (int ks = 0; ks < kPgKeys / 16; ++ks) {
            const uint64_t ad = a + ((2 * m * L::kChunkBytes + ks * 16 * 128) >> 4), bd = p_mn + ((ks * 16 * 128) >> 4);
            if (ks == 0)
              mma_f16_if<false>(on, o_tmem + N * m, ad, bd, id_pv, more);
            else
              mma_f16_if<true>(on, o_tmem + N * m, ad, bd, id_pv);
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
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax and output
    // All softmax warps take the same way: the block counts are those of a wait that succeeded for all of them, and
    // what they decide in a block is a vote over all.  So the hardware barriers, whose wait has no limit, are passed by
    // all or by none.
    const int etid = threadIdx.x - 128;
    const int quarter = warp & 3;             // tensor-memory lane quarter
    const int cb = ((warp - 4) >> 2) * kC;    // this thread's columns [cb, cb + kC)
    const int r = quarter * 32 + lane;        // row of the block (scores) / dim of a tile (output)
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float to_log2 = p.scale * 1.4426950408889634f;
    const uint64_t to_log2_2 = pack_f32x2(to_log2, to_log2), minus = pack_f32x2(-1.f, -1.f);
    uint8_t* p_row = p_s + (cb / 64) * (kPgKeys * 128);
    uint32_t gb = 0;
    uint64_t lsum[kC / 2];
    float x[kC];
    const auto load = [&](uint32_t at) {
      if constexpr (kC == 32) {
        tmem_ld_x32_sync(at, x);
      } else {
        tmem_ld_x16(at, x);
        tmem_wait_ld_regs16(x);
      }
    };
    for (int n = 0;; ++n) {
      mbar_wait(&part_full[n & 1], static_cast<uint32_t>(n >> 1) & 1u, abort_flag, err, 0xA0);
      const PagedPart part = part_s[n & 1];
      const int nb = part.blocks;
      if (etid < N) max_s[etid] = kPgNoBound;
#pragma unroll
      for (int c = 0; c < kC / 2; ++c) lsum[c] = 0ull;
      if (bar_or(kTcEpiBar, kPgSoftThreads, *abort_flag != 0)) break;
      if (part.unit < 0) break;
      const PagedUnit un = paged_unit(p, part.unit, N);
      const int* end = end_s + (n & 1) * N + cb;
      const bool used = cb < un.cols;  // (of columns that are not, nothing is read, written or kept)
      for (int b = 0; b < nb; ++b, ++gb) {
        const uint32_t slot = gb % kPgSlots;
        mbar_wait(&blk_full[slot], (gb / kPgSlots) & 1u, abort_flag, err, 0xA1);
        const PagedBlock& blk = block_s[slot];
        const bool full = blk.full != 0;
        const int row = blk.row + r;
        const int c0 = blk.c0 - cb, c1 = blk.c1 - cb;
        const bool here = ((blk.pages >> (r >> p.pages.log_rows)) & 1u) != 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&blk_empty[slot]);
        const uint32_t s_at = s_tmem + N * (gb % kSc) + lane_off + cb;
        mbar_wait(&s_full[gb % kSc], (gb / kSc) & 1u, abort_flag, err, 0xA2);
        tc_fence_after_sync();
        bool odd = false;  // a score that is no number in a block that not every column sees all of
        // scores in log2 units, minus infinity where a column does not see the row
        const unsigned span = !here ? 0u : static_cast<unsigned>(row < p.first ? INT32_MAX : p.window);
        const auto sees = [&](int c) {  // 0 <= end - 1 - row < span
          return c >= c0 && c < c1 && static_cast<unsigned>(end[c] - 1 - row) < span;
        };
        const auto masked_scores = [&]() {
          load(s_at);
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            odd |= !(fabsf(x[c]) < INFINITY);
            x[c] = sees(c) ? x[c] * to_log2 : -INFINITY;
          }
        };
        // exponents relative to the bounds
        const auto exponents = [&](bool bad) {
          if (full) {
            load(s_at);
          } else {
            masked_scores();
          }
          const uint64_t f2 = full ? to_log2_2 : pack_f32x2(1.f, 1.f);
#pragma unroll
          for (int c = 0; c < kC; c += 4) {
            const float4 mv = *reinterpret_cast<const float4*>(max_s + cb + c);
            unpack_f32x2(fma_f32x2(pack_f32x2(mv.x, mv.y), minus, fma_f32x2(pack_f32x2(x[c], x[c + 1]), f2, 0ull)), x[c], x[c + 1]);
            unpack_f32x2(fma_f32x2(pack_f32x2(mv.z, mv.w), minus, fma_f32x2(pack_f32x2(x[c + 2], x[c + 3]), f2, 0ull)), x[c + 2],
                         x[c + 3]);
          }
          if (bad) {
#pragma unroll
            for (int c = 0; c < kC; ++c) x[c] = -INFINITY;
          }
        };
        float over = -INFINITY;
        if (used) {
          exponents(false);
#pragma unroll
          for (int c = 0; c < kC; c += 2) over = max3(over, x[c], x[c + 1]);
        }
        if (bar_or(kTcEpiBar, kPgSoftThreads, over > kTcLazyLog2 || odd)) {
          // rare: a bound has to be raised, or a masked row holds what is no number
          if (gb > 0) mbar_wait(pv_done, (gb - 1) & 1u, abort_flag, err, 0xA3);
          tc_fence_after_sync();
          bool bad = false;
          if (bar_or(kTcEpiBar, kPgSoftThreads, odd)) {
            // 0 times such a value would still be no number in the weighted sum.  So a row that holds one is taken out of the
            // products, and the columns that see it get a sum that is no number.
            for (int m = 0; m < kTi; ++m) mbar_wait(&kv_full[(gb % kSt) * kTi + m], (gb / kSt) & 1u, abort_flag, err, 0xA6);
            uint8_t* at = kv_s + (gb % kSt) * L::kStageBytes + r * 128;
            for (int c = 0; c < kCh; ++c)
              for (int i = 0; i < 8; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(at + c * L::kChunkBytes + i * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) bad |= (w[k] & 0x7F80u) == 0x7F80u || (w[k] & 0x7F800000u) == 0x7F800000u;
              }
            named_bar_sync(kTcEpiBar, kPgSoftThreads);
            bad = bad && !full;  // (a full block's row is seen by all columns: what comes of it is theirs)
            if (bad) {
              if (cb == 0)
                for (int c = 0; c < kCh; ++c)
                  for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(at + c * L::kChunkBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
              const float none = __int_as_float(0x7FFFFFFF);
#pragma unroll
              for (int c = 0; c < kC; c += 2) {
                float s0, s1;
                unpack_f32x2(lsum[c / 2], s0, s1);
                lsum[c / 2] = pack_f32x2(sees(c) ? none : s0, sees(c + 1) ? none : s1);
              }
            }
          }
          // the largest scores of each column
          int* top_s = reinterpret_cast<int*>(alpha_s);
          if (etid < N) top_s[etid] = ordered(-INFINITY);
          named_bar_sync(kTcEpiBar, kPgSoftThreads);
          if (used) {
            if (full) {
              load(s_at);
#pragma unroll
              for (int c = 0; c < kC; ++c) x[c] *= to_log2;
            } else {
              masked_scores();
            }
            if (bad) {
#pragma unroll
              for (int c = 0; c < kC; ++c) x[c] = -INFINITY;
            }
            if constexpr (kC == 32) {
              xpose_reduce32(x, lane, [](float v, float w) { return fmaxf(v, w); });
              atomicMax(top_s + cb + lane, ordered(x[0]));
            } else {
              xpose_reduce16(x, lane, [](float v, float w) { return fmaxf(v, w); });
              if ((lane & 1) == 0) atomicMax(top_s + cb + (lane >> 1), ordered(x[0]));
            }
          }
          named_bar_sync(kTcEpiBar, kPgSoftThreads);
          bool moved = false;
          if (etid < N) {
            const float bm = from_ordered(top_s[etid]), mo = max_s[etid];
            const float mn = bm > mo + kTcLazyLog2 ? bm : mo;
            moved = mn != mo && mo != kPgNoBound;
            alpha_s[etid] = moved ? exp2f(mo - mn) : 1.f;
            max_s[etid] = mn;
          }
          moved = bar_or(kTcEpiBar, kPgSoftThreads, moved);
          if (moved && b > 0 && used) {
            // sums and output accumulators of earlier blocks follow (this thread: its dim of every tile, its columns)
#pragma unroll
            for (int c = 0; c < kC; c += 2)
              lsum[c / 2] = fma_f32x2(lsum[c / 2], pack_f32x2(alpha_s[cb + c], alpha_s[cb + c + 1]), 0ull);
#pragma unroll 1
            for (int m = 0; m < kTi; ++m) {
#pragma unroll
              for (int c = 0; c < kC; c += 16) {
                tmem_ld_x16(o_tmem + lane_off + N * m + cb + c, x);
                tmem_wait_ld_regs16(x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= alpha_s[cb + c + j];
                tmem_st_x16(o_tmem + lane_off + N * m + cb + c, x);
              }
            }
            tmem_wait_st();
          }
          if (used) exponents(bad);
        }
        // weights, written into the bf16 row P[row r] once the weighted sum before has read P
        if (gb > 0) mbar_wait(pv_done, (gb - 1) & 1u, abort_flag, err, 0xA4);
        if (used) {
#pragma unroll
          for (int c = 0; c < kC; c += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float e0 = exp2_approx(x[c + 2 * i]), e1 = exp2_approx(x[c + 2 * i + 1]);
              const __nv_bfloat162 w = __floats2bfloat162_rn(e0, e1);
              pk[i] = *reinterpret_cast<const uint32_t*>(&w);
              x[c + 2 * i] = e0;
              x[c + 2 * i + 1] = e1;
            }
            *reinterpret_cast<uint4*>(p_row + swz128(r, 2 * (cb % 64 + c))) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        }
        fence_proxy_async_shared();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        if (used) {
#pragma unroll
          for (int c = 0; c < kC; c += 2) lsum[c / 2] = fma_f32x2(pack_f32x2(x[c], x[c + 1]), pack_f32x2(1.f, 1.f), lsum[c / 2]);
        }
      }
      // the part's end: sums over the 128 rows (P's place holds the quarters' once it is free)
      if (nb > 0) mbar_wait(pv_done, (gb - 1) & 1u, abort_flag, err, 0xA5);
      tc_fence_after_sync();
      named_bar_sync(kTcEpiBar, kPgSoftThreads);
      float* red_s = reinterpret_cast<float*>(p_s);  // [4][N]
      {
#pragma unroll
        for (int c = 0; c < kC; c += 2) unpack_f32x2(lsum[c / 2], x[c], x[c + 1]);
        if constexpr (kC == 32) {
          xpose_reduce32(x, lane, [](float v, float w) { return v + w; });
          red_s[quarter * N + cb + lane] = x[0];
        } else {
          xpose_reduce16(x, lane, [](float v, float w) { return v + w; });
          if ((lane & 1) == 0) red_s[quarter * N + cb + (lane >> 1)] = x[0];
        }
      }
      named_bar_sync(kTcEpiBar, kPgSoftThreads);
      const int64_t row0 = static_cast<int64_t>(un.t0) * p.H + un.h0;  // the unit's first (token, head)
      const int64_t place = 2 * static_cast<int64_t>(cta) + (part.way == kPgHead ? 1 : 0);  // of a shared unit's part
      if (etid < un.cols) {
        const float l = (red_s[etid] + red_s[N + etid]) + (red_s[2 * N + etid] + red_s[3 * N + etid]);
        if (part.way == kPgWhole) {
          const int h = p.groups > 1 ? un.h0 + etid : etid % p.H;
          alpha_s[etid] = paged_factor(max_s[etid], l, p.sink, h, p.lse != nullptr ? p.lse + row0 + etid : nullptr);
        } else {
          __stcg(p.stats + place * 2 * N + etid, max_s[etid]);
          __stcg(p.stats + place * 2 * N + N + etid, l);
        }
      }
      named_bar_sync(kTcEpiBar, kPgSoftThreads);
      const bool dims = D >= 128 || quarter < 2;  // (the upper half of a 64-dim row's tile is padding)
      if (used) {
        for (int m = 0; m < kTi; ++m) {
#pragma unroll
          for (int c = 0; c < kC; c += 16) {
            float o[16];
            if (nb > 0) {
              tmem_ld_x16(o_tmem + lane_off + N * m + cb + c, o);
              tmem_wait_ld_regs16(o);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = 0.f;
            }
            if (part.way != kPgWhole) {
              if (dims) {
                float* to = p.partial + (place * N + cb + c) * D + 128 * m + r;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (cb + c + j < un.cols) __stcg(to + j * D, o[j]);
              }
              continue;
            }
            // Neighbouring lanes (dims) trade halves of a pair of columns, so that each stores two dims of one: 64
            // contiguous bytes per column and warp.
            const bool second = (lane & 1) != 0;
            uint16_t* dst = p.out + (row0 + cb + c + (second ? 1 : 0)) * D + 128 * m + (r & ~1);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 f = *reinterpret_cast<const float2*>(alpha_s + cb + c + j);
              const __nv_bfloat162 two = __floats2bfloat162_rn(o[j] * f.x, o[j + 1] * f.y);
              const uint32_t w = *reinterpret_cast<const uint32_t*>(&two);
              const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 1);
              const uint32_t own = second ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
              if (dims && cb + c + j + (second ? 1 : 0) < un.cols)
                *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(j) * D) = own;
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
      named_bar_sync(kTcEpiBar, kPgSoftThreads);  // alpha_s, max_s and P's place are written anew by the next part
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tbase, 512);
}

// ------------------------------------------------------------------------------------ shared units

constexpr int kPgJoinThreads = 128;
constexpr int kPgMaxCtas = 512;  // CTAs that may share a unit

// Joins the parts of the units that several CTAs shared: block (i, j) the columns j, j + gridDim.y, ... of the i-th entry.
template <int D>
__global__ void __launch_bounds__(kPgJoinThreads) paged_join_kernel(const PagedAttnParams p) {
  constexpr int N = paged_cols(D);
  __shared__ float w_s[kPgMaxCtas];
  __shared__ float red_s[kPgJoinThreads / 32];
  wait_stream();
  const int4 e = __ldcg(p.shared + blockIdx.x);
  const int parts = min(e.z, kPgMaxCtas);
  if (parts <= 0) return;
  const PagedUnit un = paged_unit(p, e.x, N);
  const int64_t row0 = static_cast<int64_t>(un.t0) * p.H + un.h0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // part k of the unit: the end of the first CTA's piece, the beginnings of the others'
  const auto place = [&](int k) { return 2 * (static_cast<int64_t>(e.y) + k) + (k == 0 ? 1 : 0); };
  for (int c = blockIdx.y; c < un.cols; c += gridDim.y) {
    float top = kPgNoBound;
    for (int k = threadIdx.x; k < parts; k += kPgJoinThreads) {
      const float m = __ldcg(p.stats + place(k) * 2 * N + c);
      w_s[k] = m;
      top = fmaxf(top, m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) red_s[warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red_s[0], red_s[1]), fmaxf(red_s[2], red_s[3]));
    float sum = 0.f;
    for (int k = threadIdx.x; k < parts; k += kPgJoinThreads) {
      const float m = w_s[k];
      const float f = m == kPgNoBound ? 0.f : exp2f(m - top);
      const float l = __ldcg(p.stats + place(k) * 2 * N + N + c);
      sum += l != l ? l : l * f;  // (a sum that is no number stays one, whatever its part weighs)
      w_s[k] = f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) red_s[warp] = sum;
    __syncthreads();
    sum = (red_s[0] + red_s[1]) + (red_s[2] + red_s[3]);
    const int h = p.groups > 1 ? un.h0 + c : c % p.H;
    const float f = paged_factor(top, sum, p.sink, h, p.lse != nullptr && threadIdx.x == 0 ? p.lse + row0 + c : nullptr);
    for (int d = 4 * threadIdx.x; d < D; d += 4 * kPgJoinThreads) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kAhead = 8;  // parts in flight
      for (int k0 = 0; k0 < parts; k0 += kAhead) {
        float4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + k < parts) v[k] = __ldcg(reinterpret_cast<const float4*>(p.partial + (place(k0 + k) * N + c) * D + d));
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float w = k0 + k < parts ? w_s[k0 + k] : 0.f;
          acc.x = fmaf(v[k].x, w, acc.x);
          acc.y = fmaf(v[k].y, w, acc.y);
          acc.z = fmaf(v[k].z, w, acc.z);
          acc.w = fmaf(v[k].w, w, acc.w);
        }
      }
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * f, acc.y * f), hi = __floats2bfloat162_rn(acc.z * f, acc.w * f);
      *reinterpret_cast<uint2*>(p.out + (row0 + c) * D + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    __syncthreads();
  }
}

}  // namespace dsa
