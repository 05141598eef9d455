// Rows into the 4-bit paged cache and back (the format: kv4.cuh).
//
// Write, per row of D bf16 values x:
//     r   = the smallest power of two >= 2^-100 with max|x| <= 6 * 448 * r
//     s_g = max|x in group g| / (6 r) rounded to the nearest e4m3 value, ties to even
//     c_d = x_d / (r s_g) rounded to the nearest e2m1 value, ties to even, beyond 6 to 6 (0 where s_g = 0)
// Every rounding is that of the exact quotient.  r being a power of two, x / r is exact.  For s_g the
// dividend has 8 significant bits and the borders between e4m3 values, times 6, at most 7: a quotient
// that is no border is at least 2^-9 of itself away from one, so the fp32 division cannot move it across.  For
// c_d the borders m are k / 4 (.25 to 5), m * s_g has at most 7 significant bits and x / r has 8, so x / (r s_g) is
// either equal to a border or at least 2^-8 of it, hence 2^-10, away; the product of x / r with the rounded
// reciprocal of s_g is off by less than 2^-20, and adding and subtracting 6144 rounds it to a multiple of
// 2^-11, which restores a quotient that is a border exactly and moves no other across one.
//
// HBM-bound: 2 D bytes in and D / 2 + D / 16 + 4 out per row (the reading direction the reverse).  A lane
// holds one group of 16 values (32 bytes of bf16, 8 bytes of codes, one scale byte), so a row takes
// D / 16 lanes and a warp 512 / D rows at a time, kRowSets of them with all their loads issued first.
#pragma once

#include "kv4.cuh"
#include "quant_kernel.cuh"

namespace dsa {

constexpr int kKv4CodecThreads = 256;
constexpr int kRowSets = 4;

template <int D>
__global__ void __launch_bounds__(kKv4CodecThreads) kv4_write_kernel(const uint16_t* __restrict__ x, int N,
                                                                     const int32_t* __restrict__ seq,
                                                                     const int32_t* __restrict__ pos, Kv4Pool c) {
  constexpr int kLanes = D / kKv4Group;  // lanes per row
  constexpr int kRows = 32 / kLanes;     // rows per warp and set
  const int lane = threadIdx.x & 31;
  const int sub = lane % kLanes;
  const int64_t warp0 = (static_cast<int64_t>(blockIdx.x) * kKv4CodecThreads + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (kKv4CodecThreads / 32);
  const int rows = 1 << c.log_rows;
  for (int64_t r0 = warp0 * kRows * kRowSets; r0 < N; r0 += nwarps * kRows * kRowSets) {
    uint4 raw[kRowSets][2];
    int page[kRowSets], at[kRowSets];
#pragma unroll
    for (int i = 0; i < kRowSets; ++i) {
      const int64_t row = r0 + i * kRows + lane / kLanes;
      page[i] = -1;
      at[i] = 0;
      raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (row < N) {
        const uint4* src = reinterpret_cast<const uint4*>(x + row * D + sub * kKv4Group);
        raw[i][0] = __ldcs(src);
        raw[i][1] = __ldcs(src + 1);
        at[i] = __ldg(pos + row);
        page[i] = __ldg(seq + row);
      }
    }
#pragma unroll
    for (int i = 0; i < kRowSets; ++i) {
      page[i] = kv4_page(c, page[i], at[i]);
      at[i] &= rows - 1;
    }
#pragma unroll
    for (int i = 0; i < kRowSets; ++i) {
      const uint32_t w[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                             raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
      // largest magnitudes, compared as bf16 bits
      uint32_t g = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) g = max(g, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
      uint32_t top = g;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      // 2688 = 1.3125 * 2^11: the exponent of r from the exponent and the 7 mantissa bits of max|x|
      int e = static_cast<int>(top >> 7) - 127 - ((top & 0x7Fu) <= 40u ? 11 : 10);
      e = max(e, kKv4MinExp);
      const float up = __int_as_float((127 - e) << 23);  // 1 / r
      const float gm = __uint_as_float(g << 16) * up;
      const uint32_t s8 = cvt_e4m3x2(gm / 6.0f, 0.0f) & 0xFFu;
      const uint32_t s16 = e4m3x2_to_f16x2(s8);
      const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(s16 & 0xFFFFu)));
      const float f = s > 0.0f ? up * (1.0f / s) : 0.0f;
      uint32_t codes[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xFFFF0000u);
        const float a = copysignf((fabsf(lo * f) + 6144.0f) - 6144.0f, lo);
        const float b = copysignf((fabsf(hi * f) + 6144.0f) - 6144.0f, hi);
        codes[j >> 2] |= cvt_e2m1x2(a, b) << (8 * (j & 3));
      }
      if (page[i] >= 0) {
        uint8_t* base = c.cache + static_cast<int64_t>(page[i]) * rows * kv4_row_bytes(D);
        *reinterpret_cast<uint2*>(base + at[i] * (D / 2) + sub * 8) = make_uint2(codes[0], codes[1]);
        base += rows * (D / 2);
        base[at[i] * kLanes + sub] = static_cast<uint8_t>(s8);
        if (sub == 0) reinterpret_cast<float*>(base + rows * kLanes)[at[i]] = __int_as_float((127 + e) << 23);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kKv4CodecThreads) kv4_read_kernel(uint16_t* __restrict__ out, int N,
                                                                    const int32_t* __restrict__ seq,
                                                                    const int32_t* __restrict__ pos, Kv4Pool c) {
  constexpr int kLanes = D / kKv4Group;
  constexpr int kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int sub = lane % kLanes;
  const int64_t warp0 = (static_cast<int64_t>(blockIdx.x) * kKv4CodecThreads + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (kKv4CodecThreads / 32);
  const int rows = 1 << c.log_rows;
  for (int64_t r0 = warp0 * kRows * kRowSets; r0 < N; r0 += nwarps * kRows * kRowSets) {
    int page[kRowSets], at[kRowSets];
    uint2 raw[kRowSets];
    uint32_t s8[kRowSets];
    float r[kRowSets];
#pragma unroll
    for (int i = 0; i < kRowSets; ++i) {
      const int64_t row = r0 + i * kRows + lane / kLanes;
      page[i] = row < N ? __ldg(seq + row) : -1;
      at[i] = row < N ? __ldg(pos + row) : 0;
    }
#pragma unroll
    for (int i = 0; i < kRowSets; ++i) {
      page[i] = kv4_page(c, page[i], at[i]);
      at[i] &= rows - 1;
    }
#pragma unroll
    for (int i = 0; i < kRowSets; ++i) {
      raw[i] = make_uint2(0u, 0u);
      s8[i] = 0u;
      r[i] = 0.0f;
      if (page[i] >= 0) {
        const uint8_t* base = c.cache + static_cast<int64_t>(page[i]) * rows * kv4_row_bytes(D);
        raw[i] = *reinterpret_cast<const uint2*>(base + at[i] * (D / 2) + sub * 8);
        base += rows * (D / 2);
        s8[i] = base[at[i] * kLanes + sub];
        r[i] = reinterpret_cast<const float*>(base + rows * kLanes)[at[i]];
      }
    }
#pragma unroll
    for (int i = 0; i < kRowSets; ++i) {
      const int64_t row = r0 + i * kRows + lane / kLanes;
      if (row >= N) continue;
      const uint32_t s = e4m3x2_to_f16x2(s8[i] | (s8[i] << 8));
      uint32_t o[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[4];
        e2m1x8_to_f16x2(h == 0 ? raw[i].x : raw[i].y, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t p = hmul2(v[j], s);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
          const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * r[i], f.y * r[i]);
          o[4 * h + j] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(out + row * D + sub * kKv4Group);
      __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
      __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
    }
  }
}

}  // namespace dsa
