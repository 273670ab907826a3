// Device helpers that the attention kernels share: matrix products of 16-bit elements, rows of
// keys and values in shared memory, the weights' range.
#pragma once

#include "ops_device.hpp"

namespace tf_exl3 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (DT == TF_DT_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Matrix products and reads of shared memory stay on their side; other work may cross.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x2 | 0x4 | 0x10); }

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == TF_DT_F16) {
    const half2_t h = {(_Float16)lo, (_Float16)hi};
    return __builtin_bit_cast(uint32_t, h);
  } else {
    const f32x2 f = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
  }
}

// The four lane groups' values of a row (lanes l, l + 16, l + 32, l + 48), joined.
__device__ __forceinline__ float groups_max(float v) {
  u32x2 s = __builtin_amdgcn_permlane16_swap(f32_to_bits(v), f32_to_bits(v), false, false);
  v = fmaxf(bits_to_f32(s[0]), bits_to_f32(s[1]));
  s = __builtin_amdgcn_permlane32_swap(f32_to_bits(v), f32_to_bits(v), false, false);
  return fmaxf(bits_to_f32(s[0]), bits_to_f32(s[1]));
}
__device__ __forceinline__ float groups_sum(float v) {
  u32x2 s = __builtin_amdgcn_permlane16_swap(f32_to_bits(v), f32_to_bits(v), false, false);
  v = bits_to_f32(s[0]) + bits_to_f32(s[1]);
  s = __builtin_amdgcn_permlane32_swap(f32_to_bits(v), f32_to_bits(v), false, false);
  return bits_to_f32(s[0]) + bits_to_f32(s[1]);
}

// A row's weights for the second product are 2^(x - base + kUp), its base at most kSlack below its
// largest score so far. They are rounded to the inputs' 16 bits, half an ulp each, because that product's operands have no more (their
// sum is taken before, in fp32): errors against 64 bits are 1.1 to 1.4 times those of weights in fp32. bf16 has fp32's exponents. fp16 begins at 2^-14 and ends at 2^16: a base that stands
// for 2^13 keeps half a unit in the last place down to 2^-27 of the row's largest weight, and 2^-38 of that below
// (half a step of the subnormals). Slacks of 2^8, 2^4, 2^3, 2^2 and 1 with the room used up, fp16, us: 64-node trees
// 65.7 / 65.5 / 66.0 / 67.4 / 71.9, 32 x 16 nodes over 16384 positions 394 to 396 for all.
template <int DT>
struct Weights {
  static constexpr float kUp = DT == TF_DT_F16 ? 13.f : 0.f, kSlack = DT == TF_DT_F16 ? 2.f : 8.f;
};

// Shared memory holds rows of DP elements in 16-byte chunks; chunk c of row r stands at
// c ^ (a function of r), so that neither the 16 rows x 16 bytes that a matrix operand of keys
// takes at once nor the 8 rows x 32 bytes of a transposing load meet in a bank.
template <int DP>
__device__ __forceinline__ int key_chunk(int r, int c) { return c ^ (DP == 64 ? (r >> 1) & 7 : r & 15); }
template <int DP>
__device__ __forceinline__ int value_chunk(int r, int c) { return c ^ (DP == 64 ? ((r >> 1) & 3) << 1 : (r & 7) << 1); }

// Four neighbouring columns' worth of 16-bit infinities and NaN to zero; whether any was.
template <int DT>
__device__ __forceinline__ bool drop_nonfinite(u32x4& v) {
  constexpr uint32_t top = DT == TF_DT_F16 ? 0x7C00u : 0x7F80u;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u = v[i];
    if ((u & top) == top) u &= 0xFFFF0000u, any = true;
    if ((u & top << 16) == top << 16) u &= 0xFFFFu, any = true;
    v[i] = u;
  }
  return any;
}

}  // namespace tf_exl3
