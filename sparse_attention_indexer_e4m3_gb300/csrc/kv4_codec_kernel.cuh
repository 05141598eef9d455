// Rows into the 4-bit paged cache and back (the format: kv4.cuh).
//
// Write, per row of D bf16 values x:
//     r   = the smallest power of two >= 2^-100 with max|x| <= 6 * 448 * r
//     s_g = max|x in group g| / (6 r) rounded to the nearest e4m3 value, ties to even
//     c_d = x_d / (r s_g) rounded to the nearest e2m1 value, ties to even, beyond 6 to 6 (0 where s_g = 0)
// Every rounding is that of the exact quotient, without a division.  r being a power of two, x / r is exact.
// A quotient of two numbers of at most 8 significant bits that is not equal to a third of that kind is at least
// 2^-9 of itself away from it: cross-multiplied, both sides are whole numbers of at most 16 bits.  max|x| has
// 8 significant bits and the borders between e4m3 values, times 6, at most 7, so max|x| / (6 r) is either on a
// border or 2^-9 away from it; as product with the rounded 1 / 6 it is off by less than 2^-22, and rounded to
// 12 bits it lands on the border exactly where it was on it and else stays on its side.  The borders m between
// the codes are k / 4 (.25 to 5), m s_g has at most 7 bits and x / r has 8, so x / (r s_g) is either a border or
// at least 2^-8 of it, hence 2^-10, away; the reciprocal of s_g is off by at most 2^-23, and adding 6144 rounds
// the product to a multiple of 2^-11, which again restores a border exactly and moves nothing across one.
//
// Memory-bound: 2 D bytes in and D / 2 + D / 16 + 4 out per row (the reading direction the reverse); 1048576 rows of 512
// 250 us to write (5.5 TB/s) and 265 to read (5.2), 65536 rows, which L2 mostly holds, 15.6 and 14.0.  A lane
// holds one group of 16 values (32 bytes of bf16 in one access, 8 bytes of codes, one scale byte), so a row takes
// D / 16 lanes and a warp 512 / D rows.  One group per thread and many threads: two to eight groups per thread
// with their loads issued first took 5 to 25% longer at 20011 to 65536 rows, and longer still at 61.
#pragma once

#include "kv4.cuh"
#include "quant_kernel.cuh"

namespace dsa {

constexpr int kKv4CodecThreads = 256;

// 32 contiguous bytes (32-byte aligned) in one access, not kept in L1.
__device__ __forceinline__ void ld_32(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The larger of two non-negative bf16 values, in both halves.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Rounded to 12 significant bits (finite, not at the top of the range).
__device__ __forceinline__ float round_12bits(float x) { return __uint_as_float((__float_as_uint(x) + 0x800u) & 0xFFFFF000u); }
template <int D>
__global__ void __launch_bounds__(kKv4CodecThreads) kv4_write_kernel(const uint16_t* x, int N,
                                                                     const int32_t* seq, const int32_t* pos,
                                                                     const int32_t* lacking, Kv4Pool c) {
  constexpr int kLanes = D / kKv4Group;  // lanes per row
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kKv4CodecThreads + threadIdx.x) / kLanes;
  const int sub = threadIdx.x % kLanes;
  const int rows = 1 << c.log_rows;
  uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  int page = -1, at = 0;
  wait_stream();
  if (row < N) {
    const int short_of = lacking != nullptr ? ld_after_wait(lacking) : 0;
    at = ld_after_wait(pos + row);
    page = ld_after_wait(seq + row);
    ld_32(x + row * D + sub * kKv4Group, w);
    page = kv4_page(c, page, at);
    at &= rows - 1;
    if (short_of != 0) page = -1;
  }
  // largest magnitudes, as bf16 bits
  uint32_t both = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) both = max_bf16x2(both, w[j] & 0x7FFF7FFFu);
  const uint32_t g = max(both & 0xFFFFu, both >> 16);
  uint32_t top = g;
  if constexpr (kLanes == 32) {
    top = __reduce_max_sync(0xffffffffu, top);
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (page < 0) return;
  // 2688 = 1.3125 * 2^11: the exponent of r from the exponent and the 7 mantissa bits of max|x|
  int e = static_cast<int>(top >> 7) - 127 - ((top & 0x7Fu) <= 40u ? 11 : 10);
  e = max(e, kKv4MinExp);
  const float up = __int_as_float((127 - e) << 23);  // 1 / r
  const float gm = __uint_as_float(g << 16) * up;
  const uint32_t s8 = cvt_e4m3x2(round_12bits(gm * (1.0f / 6.0f)), 0.0f) & 0xFFu;
  const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(s8) & 0xFFFFu)));
  const float f = s > 0.0f ? up * rcp_approx(s) : 0.0f;
  uint32_t codes[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = __uint_as_float(w[4 * i + j] << 16), hi = __uint_as_float(w[4 * i + j] & 0xFFFF0000u);
      v[2 * j] = copysignf(fmaf(fabsf(lo), f, 6144.0f) - 6144.0f, lo);
      v[2 * j + 1] = copysignf(fmaf(fabsf(hi), f, 6144.0f) - 6144.0f, hi);
    }
    codes[i] = cvt_e2m1x8(v);
  }
  uint8_t* base = c.cache + static_cast<int64_t>(page) * rows * kv4_row_bytes(D);
  *reinterpret_cast<uint2*>(base + at * (D / 2) + sub * 8) = make_uint2(codes[0], codes[1]);
  base += rows * (D / 2);
  base[at * kLanes + sub] = static_cast<uint8_t>(s8);
  if (sub == 0) reinterpret_cast<float*>(base + rows * kLanes)[at] = __int_as_float((127 + e) << 23);
}

template <int D>
__global__ void __launch_bounds__(kKv4CodecThreads) kv4_read_kernel(uint16_t* out, int N,
                                                                    const int32_t* seq,
                                                                    const int32_t* pos, Kv4Pool c) {
  constexpr int kLanes = D / kKv4Group;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kKv4CodecThreads + threadIdx.x) / kLanes;
  const int sub = threadIdx.x % kLanes;
  wait_stream();
  if (row >= N) return;
  const int rows = 1 << c.log_rows;
  int at = ld_after_wait(pos + row);
  const int page = kv4_page(c, ld_after_wait(seq + row), at);
  at &= rows - 1;
  uint2 raw = make_uint2(0u, 0u);
  uint32_t s8 = 0u;
  float r = 0.0f;
  if (page >= 0) {
    const uint8_t* base = c.cache + static_cast<int64_t>(page) * rows * kv4_row_bytes(D);
    raw = *reinterpret_cast<const uint2*>(base + at * (D / 2) + sub * 8);
    base += rows * (D / 2);
    s8 = base[at * kLanes + sub];
    r = reinterpret_cast<const float*>(base + rows * kLanes)[at];
  }
  const uint32_t s = e4m3x2_to_f16x2(s8 | (s8 << 8));
  uint32_t o[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[4];
    e2m1x8_to_f16x2(h == 0 ? raw.x : raw.y, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t p = hmul2(v[j], s);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * r, f.y * r);
      o[4 * h + j] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  st_32(out + row * D + sub * kKv4Group, o);
}

}  // namespace dsa
