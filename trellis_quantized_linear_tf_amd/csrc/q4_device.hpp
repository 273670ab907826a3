// A cache's rows in 4 bits: groups of 32 numbers, each number 0 .. 15 times the group's scale
// plus its minimum, both fp16. Codes of eight numbers are a word whose nibbles i and i + 4 are the
// numbers 2i and 2i + 1: shifted by 4i and masked, a word holds a pair where a pair of 16-bit
// elements holds it.
#pragma once

#include "ops_device.hpp"

namespace tf_exl3 {

constexpr int kQ4Group = 32;
// Of a number's magnitude: a scale that was rounded up takes the largest code of numbers within +-M to
// M (1 + 2^-10), which has to stay below 65520, where fp16 rounds to infinity.
constexpr float kQ4Most = 65408.f;

typedef u32x4 u32x4_word __attribute__((aligned(4)));  // codes begin at any word

// Scale and minimum of a group, as they stand in the cache.
struct Q4Pair {
  float scale, low;
};

__device__ __forceinline__ Q4Pair q4_unpack(uint32_t pair) {
  return {f16_bits_to_f32((uint16_t)pair), f16_bits_to_f32((uint16_t)(pair >> 16))};
}

// The values of a word's eight codes in fp32. A pair of codes, masked where it stands, is a pair of fp16
// subnormals, code * 2^-24 or, 4 bits up, code * 2^-20, which the mixed multiply-add takes as they are;
// the scales make up for it (their products with codes are exact in fp32).
__device__ __forceinline__ void q4_values(uint32_t word, Q4Pair p, float (&x)[8]) {
  const float scales[2] = {p.scale * 16777216.f, p.scale * 1048576.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = (i < 2 ? word : word >> 8) & (i % 2 ? 0x00F000F0u : 0x000F000Fu);
    const half2_t h = __builtin_bit_cast(half2_t, t);
    x[2 * i] = __builtin_fmaf((float)h[0], scales[i % 2], p.low);
    x[2 * i + 1] = __builtin_fmaf((float)h[1], scales[i % 2], p.low);
  }
}

// Eight values as a 16-byte piece of a row of DT. fp16: the codes in the last bits of 1024 or, 4 bits up,
// of 64, less that, times the scale plus the minimum with one rounding.
template <int DT>
__device__ __forceinline__ u32x4 q4_piece(uint32_t word, uint32_t pair) {
  u32x4 v;
  if constexpr (DT == TF_DT_F16) {
    const half2_t h = __builtin_bit_cast(half2_t, pair);
    const half2_t scale = {h[0], h[0]}, low = {h[1], h[1]};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t bits = (i < 2 ? word : word >> 8) & (i % 2 ? 0x00F000F0u : 0x000F000Fu);
      const uint32_t base = i % 2 ? 0x54005400u : 0x64006400u;
      const half2_t n = __builtin_bit_cast(half2_t, bits | base) - __builtin_bit_cast(half2_t, base);
      v[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(n, scale, low));
    }
  } else {
    float x[8];
    q4_values(word, q4_unpack(pair), x);
    v = Elem<DT>::pack(x);
  }
  return v;
}

}  // namespace tf_exl3
