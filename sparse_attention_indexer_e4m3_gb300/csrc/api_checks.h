// Checks of arguments that the paged caches' entry points share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/dsa.h"

namespace dsa {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// Whether n elements at a and m at b, of their types' sizes, have a byte in common (what a kernel writes while it reads the other).
template <class A, class B>
bool overlap(const A* a, int64_t n, const B* b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return n > 0 && m > 0 && x < y + static_cast<uintptr_t>(m) * sizeof(B) && y < x + static_cast<uintptr_t>(n) * sizeof(A);
}
inline bool paged_d(int D) { return D == 64 || D == 128 || D == 256 || D == 512; }
inline bool paged_rows(int rows) { return rows >= 16 && rows <= 256 && (rows & (rows - 1)) == 0; }
inline int log2_of(int rows) {
  int l = 0;
  while ((1 << l) < rows) ++l;
  return l;
}
inline dsa_status done(cudaError_t e) { return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

}  // namespace dsa
