// The bf16 paged kv cache: parameters of its kernels.  Row pos of sequence r is row pos % page_rows of page
// table[r][pos / page_rows]; a page is page_rows rows of D bf16 values, each both key and value.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace dsa {

// The table that gives each sequence its pages.
struct PageTable {
  const int32_t* table;  // [R][M] page ids; anything outside [0, P) is no page
  int P, R, M;
  int log_rows;          // log2 of the page's rows
};

struct StepMapArgs {
  const int32_t* held;   // [R]
  const int32_t* added;  // [R]
  int R, T;
  int32_t* seq;          // [T] each
  int32_t* pos;
  int32_t* ks;
  int32_t* ke;
};

// How the (token, head) rows of a call are cut into units.
struct PagedCut {
  int rows;    // of a unit
  int groups;  // units of a token, where a token's heads take several of their own; else 1
  int units;
};

struct PagedAttnParams {
  PageTable pages;
  const int32_t* seq;   // [T]
  const int32_t* pos;   // [T]
  const float* sink;    // [H] or null
  uint16_t* out;        // [T][H][D] bf16
  float* lse;           // [T][H] or null
  float* partial;       // [2 CTAs][N][D] partial outputs of units that several CTAs share
  float* stats;         // [2 CTAs][2][N] their bounds and sums
  int4* shared;         // [min(units, CTAs)] the shared units: first row of q, first CTA, CTAs (0: none), rows
  int T, H;
  PagedCut whole;       // whole tokens, or a token's heads in equal units of their own
  PagedCut any;         // units wherever they begin (as `whole` where there is no choice)
  int guess;            // the cut to begin with: 0 whole, 1 any
  float per_token;      // walks over a sequence's rows that the second cut takes more than the first: for each token,
  float per_run;        // and for each run of tokens of one sequence
  int window;           // rows that a token sees up to its own
  int first;            // first rows that stay visible
  int box_rows;         // rows of one copy: those of a page, at most a block's
  alignas(8) float to_log2[2];  // the softmax scale in log2 units, twice
  uint32_t h_mul;       // n / H = (mulhi(n, h_mul) + n) >> h_shift for 0 <= n < 2^31 (set_heads)
  int h_shift;

  // 2^h_shift >= H > 2^(h_shift - 1) and h_mul = floor(2^32 (2^h_shift - H) / H) + 1: the quotient's multiplier 2^32 + h_mul lies
  // above 2^(32 + h_shift) / H by at most 1, which is too little to reach the next whole number for n < 2^32.
  void set_heads(int heads) {
    H = heads;
    h_shift = 0;
    while ((static_cast<int64_t>(1) << h_shift) < heads) ++h_shift;
    h_mul = static_cast<uint32_t>((((static_cast<uint64_t>(1) << h_shift) - heads) << 32) / heads + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int by_H(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), h_mul) + static_cast<uint32_t>(n)) >> h_shift);
  }
  __device__ __forceinline__ int head(int n) const { return n - by_H(n) * H; }
#endif
};

struct VerifyArgs {
  const float* target;    // [R][G + 1][V]
  const float* draft;     // [R][G][V]
  const int32_t* tokens;  // [R][G]
  const int32_t* count;   // [R]
  const float* u;         // [R][G + 1]
  int R, G, V;
  int32_t* accepted;      // [R]
  int32_t* token;         // [R]
};

}  // namespace dsa
