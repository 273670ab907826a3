// Device helpers of the operators around the projection: element types, 16-byte pieces
// of rows, wave and workgroup reductions in a fixed order.
#pragma once

#include <hip/hip_runtime.h>

#include "exl3_device.hpp"
#include "tf_exl3.h"

namespace tf_exl3 {

// 16 bytes of a row, at any alignment of whole elements: gfx950 loads and stores
// unaligned vectors whole, and the cache lines that two pieces share come from L1.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_elem __attribute__((aligned(2)));

__device__ __forceinline__ u32x4 load_piece(const void* p) { return *static_cast<const u32x4_elem*>(p); }
__device__ __forceinline__ void store_piece(void* p, u32x4 v) { *static_cast<u32x4_elem*>(p) = v; }

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Elements of a row of type DT as fp32 (exact for all three types), single and by the
// piece; fp32 -> DT rounds to nearest even.
template <int DT>
struct Elem;

template <>
struct Elem<TF_DT_F32> {
  typedef float type;
  static constexpr int kPiece = 4;
  static constexpr uint32_t kMinusInf = 0xFF800000u;  // a piece's dword of -inf
  __device__ static float load(float v) { return v; }
  __device__ static float store(float v) { return v; }
  __device__ static void unpack(u32x4 v, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = bits_to_f32(v[i]);
  }
  __device__ static u32x4 pack(const float (&x)[4]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f32_to_bits(x[i]);
    return v;
  }
};

template <>
struct Elem<TF_DT_F16> {
  typedef uint16_t type;
  static constexpr int kPiece = 8;
  static constexpr uint32_t kMinusInf = 0xFC00FC00u;
  __device__ static float load(uint16_t v) { return f16_bits_to_f32(v); }
  __device__ static uint16_t store(float v) { return f32_to_f16_bits(v); }
  __device__ static void unpack(u32x4 v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = v[i];  // a bit_cast of the element itself takes element 0
      const half2_t h = __builtin_bit_cast(half2_t, u);
      x[2 * i] = (float)h[0];
      x[2 * i + 1] = (float)h[1];
    }
  }
  __device__ static u32x4 pack(const float (&x)[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const half2_t h = {(_Float16)x[2 * i], (_Float16)x[2 * i + 1]};
      v[i] = __builtin_bit_cast(uint32_t, h);
    }
    return v;
  }
};

template <>
struct Elem<TF_DT_BF16> {
  typedef uint16_t type;
  static constexpr int kPiece = 8;
  static constexpr uint32_t kMinusInf = 0xFF80FF80u;
  __device__ static float load(uint16_t v) { return bf16_bits_to_f32(v); }
  __device__ static uint16_t store(float v) { return f32_to_bf16_bits(v); }
  __device__ static void unpack(u32x4 v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bits_to_f32(v[i] << 16);
      x[2 * i + 1] = bits_to_f32(v[i] & 0xFFFF0000u);
    }
  }
  __device__ static u32x4 pack(const float (&x)[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 f = {x[2 * i], x[2 * i + 1]};
      v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
    }
    return v;
  }
};

// Eight elements of a row, at any alignment of whole ones.
template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::type* p, float (&x)[8]) {
  if constexpr (DT == TF_DT_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 v = load_piece(p + 4 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * h + i] = bits_to_f32(v[i]);
    }
  } else {
    Elem<DT>::unpack(load_piece(p), x);
  }
}

template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::type* p, const float (&x)[8]) {
  if constexpr (DT == TF_DT_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      store_piece(p + 4 * h, u32x4{f32_to_bits(x[4 * h]), f32_to_bits(x[4 * h + 1]), f32_to_bits(x[4 * h + 2]),
                                   f32_to_bits(x[4 * h + 3])});
  } else {
    store_piece(p, Elem<DT>::pack(x));
  }
}

__device__ __forceinline__ float load_elem(const void* p, int dtype, int64_t i) {
  if (dtype == TF_DT_F32) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return dtype == TF_DT_F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
}

// n / d for 0 <= n < 2^31 by a product: with 2^s >= d, m = ceil(2^(31 + s) / d) exceeds the
// true factor by less than 2^s / 2^(31 + s) of n's range, so the quotient is exact.
struct FastDiv {
  uint32_t m;
  int shift;
  __device__ __forceinline__ int div(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> shift); }
};

inline FastDiv fast_div(int d) {
  int s = 0;
  while ((1ll << s) < d) ++s;
  return {(uint32_t)(((1ull << (31 + s)) + (uint64_t)d - 1) / (uint64_t)d), 31 + s};
}

// Lane l's value from the lane that a DPP control word names; `rest` where it names none or
// the row of 16 lanes is not in ROWS. A register move, where a shuffle is a trip to LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v, float rest) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, rest), __builtin_bit_cast(int, v), CTRL,
                                                               ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int v, int rest) {
  return __builtin_amdgcn_update_dpp(rest, v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double v, double rest) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const i32x2 a = __builtin_bit_cast(i32x2, v), r = __builtin_bit_cast(i32x2, rest);
  const i32x2 d = {__builtin_amdgcn_update_dpp((int)r[0], (int)a[0], CTRL, ROWS, 0xF, false),
                   __builtin_amdgcn_update_dpp((int)r[1], (int)a[1], CTRL, ROWS, 0xF, false)};
  return __builtin_bit_cast(double, d);
}

constexpr int kShr = 0x110;      // + n: n lanes up within a row of 16
constexpr int kBcast15 = 0x142;  // a row's last lane to the next row
constexpr int kBcast31 = 0x143;  // lane 31 to the upper half

__device__ __forceinline__ float lane_of(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const i32x2 a = __builtin_bit_cast(i32x2, v);
  const i32x2 d = {__builtin_amdgcn_readlane((int)a[0], lane), __builtin_amdgcn_readlane((int)a[1], lane)};
  return __builtin_bit_cast(double, d);
}

// Running sum over the wave's lanes, each lane's own value in it.
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
  v += dpp<kShr + 1, 0xF>(v, (T)0);
  v += dpp<kShr + 2, 0xF>(v, (T)0);
  v += dpp<kShr + 4, 0xF>(v, (T)0);
  v += dpp<kShr + 8, 0xF>(v, (T)0);
  v += dpp<kBcast15, 0xA>(v, (T)0);
  v += dpp<kBcast31, 0xC>(v, (T)0);
  return v;
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
  return lane_of(wave_scan(v), 63);
}

__device__ __forceinline__ float wave_max(float v) {
  constexpr float none = -__builtin_inff();
  v = fmaxf(v, dpp<kShr + 1, 0xF>(v, none));
  v = fmaxf(v, dpp<kShr + 2, 0xF>(v, none));
  v = fmaxf(v, dpp<kShr + 4, 0xF>(v, none));
  v = fmaxf(v, dpp<kShr + 8, 0xF>(v, none));
  v = fmaxf(v, dpp<kBcast15, 0xA>(v, none));
  v = fmaxf(v, dpp<kBcast31, 0xC>(v, none));
  return lane_of(v, 63);
}

// Sum and maximum over a workgroup of WAVES waves; every thread gets the result.
// `slot` is WAVES entries of shared memory, free again after the call's last barrier.
template <int WAVES, typename T>
__device__ __forceinline__ T block_sum(T v, T* slot) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  T s = slot[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) s += slot[w];
  return s;
}

template <int WAVES>
__device__ __forceinline__ float block_max(float v, float* slot) {
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = slot[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) s = fmaxf(s, slot[w]);
  return s;
}

}  // namespace tf_exl3
