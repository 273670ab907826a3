// Argument checks that the operators' C ABI shares: pointers, strides, extents, caches.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "tf_exl3.h"

namespace tf_exl3 {

constexpr int kMaxBatch = 65535;  // sequences, a grid dimension
constexpr int64_t kMaxStride = 1ll << 40;

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

inline size_t elem_size(int dt) { return dt == TF_DT_F32 ? 4 : 2; }

inline bool dtype_ok(int dt) { return dt == TF_DT_F32 || dt == TF_DT_F16 || dt == TF_DT_BF16; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (na == 0 || nb == 0 || a == nullptr || b == nullptr) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

// Bytes from the first to past the last element of [n0][n1][n2][d] with strides s.
inline size_t extent(int64_t n0, int64_t n1, int64_t n2, int64_t d, const int64_t* s, size_t elem) {
  return (size_t)((n0 - 1) * s[0] + (n1 - 1) * s[1] + (n2 - 1) * s[2] + d) * elem;
}

// A stride over a dimension of 1 is never used, whatever it is.
inline void settle(int64_t n0, int64_t n1, int64_t n2, int64_t* s) {
  if (n0 <= 1) s[0] = 0;
  if (n1 <= 1) s[1] = 0;
  if (n2 <= 1) s[2] = 0;
}

inline bool strides_ok(const int64_t* s, int64_t multiple) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] > kMaxStride || s[i] % multiple != 0) return false;
  return true;
}

// Rows that are written may not share elements: no stride of 0 over more than one of them.
inline bool apart(int64_t n0, int64_t n1, int64_t n2, const int64_t* s) {
  return (n0 <= 1 || s[0] != 0) && (n1 <= 1 || s[1] != 0) && (n2 <= 1 || s[2] != 0);
}

inline int cache_sizes(int pages, int page_size, int table_pages, int64_t table_stride) {
  if (pages < 1 || page_size < 1 || table_pages < 0 || table_stride < 0 || table_stride > kMaxStride) return TF_E_SIZE;
  // Positions are 32-bit: room for the longest sequence and its new tokens.
  if ((int64_t)table_pages * page_size > (1ll << 30)) return TF_E_SIZE;
  return TF_OK;
}

// Bytes of a row of the cache in 4 bits: codes, then scale and minimum of each 32 numbers.
inline int64_t q4_bytes(int head_dim) { return (int64_t)head_dim / 8 * 5; }

}  // namespace tf_exl3
