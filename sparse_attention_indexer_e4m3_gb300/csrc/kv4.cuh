// The 4-bit paged kv cache: layout of a page, where a row of a sequence lives, and the conversions
// between held rows and fp16 / fp32 values.
//
// A row x of D values is held as x[d] ~= r * s[d / 16] * c[d]: c[d] an e2m1 value (0, .5, 1, 1.5, 2, 3, 4,
// 6 with a sign; even d in the low half of its byte), s an unsigned e4m3 scale per 16 values, r an
// fp32 scale per row.  A page of B rows is its rows' codes [B][D / 2], then their group scales
// [B][D / 16], then their row scales [B].  s * c has at most 6 significant bits and lies between
// 2^-10 and 2688, so it is exact in fp16; the tensor-core attention works on s * c.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace dsa {

constexpr int kKv4Group = 16;      // values per e4m3 scale
constexpr int kKv4MinExp = -100;   // smallest exponent of a row scale that the quantiser writes

// Waits until the work before this kernel in its stream is complete and visible; nothing in global memory is
// touched before it.
__device__ __forceinline__ void wait_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// An ordinary load.  Not __ldg, and no const __restrict__ parameters: those promise memory that does not change while
// the kernel runs, and a kernel that starts before the work it waits for is done may not promise that (the
// compiler could move such a load ahead of wait_stream()).
template <class T>
__device__ __forceinline__ T ld_after_wait(const T* p) {
  return *p;
}

// Bytes of a held row of D values: codes, group scales, row scale.
__host__ __device__ constexpr int kv4_row_bytes(int D) { return D / 2 + D / kKv4Group + 4; }

// A pool of pages and the table that gives each sequence its pages.
struct Kv4Pool {
  uint8_t* cache;         // [P][page_rows * kv4_row_bytes(D)]
  const int32_t* table;   // [R][M] page ids; anything outside [0, P) is no page
  int P, R, M;
  int log_rows;           // log2 of the page's rows
};

struct AttnKv4Params {
  const uint16_t* q;      // [T][H][D] bf16
  Kv4Pool pool;
  const int32_t* seq;     // [T]
  const int32_t* start;   // [T] or null: list entry minus start = row of the sequence
  const float* sink;      // [H] or null
  const int32_t* idx;     // [T][K]
  uint16_t* out;          // [T][H][D] bf16
  float* lse;             // [T][H] or null
  float* partial;         // [unit][share][64][D] partial outputs where a list is shared
  float* partial_stats;   // [unit][share][2][64] their bounds and sums
  int T, H, K;
  int groups;             // ceil(H / 64)
  float scale;
};

struct ReserveArgs {
  int32_t* table;
  int32_t* ref;
  const int32_t* begin;
  const int32_t* end;
  int R, M, P, log_rows;
  int32_t* src;     // [2 R]
  int32_t* dst;     // [2 R]
  int32_t* lacking; // [1]
  int32_t* fresh;   // workspace [P]: the k-th page handed out
  int32_t* left;    // workspace [P]: the shared page it replaces, or -1
};

struct CompactArgs {
  int32_t* ref;
  int P;
  int32_t* src;    // [P / 2]
  int32_t* dst;    // [P / 2]
  int32_t* n_live; // [1]
  int32_t* remap;  // workspace [P]: new id of each page, -1 for a free one
  int32_t* table;  // [entries], relabelled by the same kernel where it is small, else null
  int entries;
};

// Page of row `pos` of sequence `seq`, or -1 where there is none.
__device__ __forceinline__ int kv4_page(const Kv4Pool& c, int seq, int pos) {
  if (static_cast<unsigned>(seq) >= static_cast<unsigned>(c.R) || pos < 0 || (pos >> c.log_rows) >= c.M) return -1;
  const int page = ld_after_wait(c.table + static_cast<int64_t>(seq) * c.M + (pos >> c.log_rows));
  return static_cast<unsigned>(page) < static_cast<unsigned>(c.P) ? page : -1;
}

// The eight e2m1 codes of a word to four fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}

// Two e4m3 codes (low byte first) to two fp16 values.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// Eight floats to the eight e2m1 codes of a word (nearest, ties to even, saturating; the first in the low bits).
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// 1 / x of a normal number, off by at most 2^-23 of it.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace dsa
