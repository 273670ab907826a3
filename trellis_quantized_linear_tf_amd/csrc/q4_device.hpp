// A cache's rows in 4 bits: groups of 32 numbers, each number 0 .. 15 times the group's scale
// plus its minimum, both fp16. Codes of eight numbers are a word whose nibbles i and i + 4 are the
// numbers 2i and 2i + 1: shifted by 4i and masked, a word holds a pair where a pair of 16-bit
// elements holds it.
#pragma once

#include "ops_device.hpp"

namespace tf_exl3 {

constexpr int kQ4Group = 32;
constexpr float kQ4Most = 65504.f;  // of a number's magnitude: fp16's largest

typedef u32x4 u32x4_word __attribute__((aligned(4)));  // codes begin at any word

// Scale and minimum of a group, as they stand in the cache.
struct Q4Pair {
  float scale, low;
};

__device__ __forceinline__ Q4Pair q4_unpack(uint32_t pair) {
  return {f16_bits_to_f32((uint16_t)pair), f16_bits_to_f32((uint16_t)(pair >> 16))};
}

// The values of a word's eight codes in fp32. A pair of codes is a pair of fp16 subnormals, code * 2^-24, which the mixed multiply-add
// takes as they are; the scale makes up for it (its products with codes are exact in fp32).
__device__ __forceinline__ void q4_values(uint32_t word, Q4Pair p, float (&x)[8]) {
  const float scale = p.scale * 16777216.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = (word >> 4 * i) & 0x000F000Fu;
    const half2_t h = __builtin_bit_cast(half2_t, t);
    x[2 * i] = __builtin_fmaf((float)h[0], scale, p.low);
    x[2 * i + 1] = __builtin_fmaf((float)h[1], scale, p.low);
  }
}

// Eight values as a 16-byte piece of a row of DT. fp16: 1024 + code in the last bits of an fp16,
// less 1024, times the scale plus the minimum with one rounding.
template <int DT>
__device__ __forceinline__ u32x4 q4_piece(uint32_t word, uint32_t pair) {
  u32x4 v;
  if constexpr (DT == TF_DT_F16) {
    const half2_t h = __builtin_bit_cast(half2_t, pair);
    const half2_t scale = {h[0], h[0]}, low = {h[1], h[1]}, base = {(_Float16)1024, (_Float16)1024};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t t = ((word >> 4 * i) & 0x000F000Fu) | 0x64006400u;
      v[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2_t, t) - base, scale, low));
    }
  } else {
    float x[8];
    q4_values(word, q4_unpack(pair), x);
    v = Elem<DT>::pack(x);
  }
  return v;
}

}  // namespace tf_exl3
