// Device helpers of the operators around the projection: element types, wave and
// workgroup reductions in a fixed order.
#pragma once

#include <hip/hip_runtime.h>

#include "exl3_device.hpp"
#include "tf_exl3.h"

namespace tf_exl3 {

// Element of a row of type DT as fp32 (exact for all three types).
template <int DT>
struct Elem;
template <>
struct Elem<TF_DT_F32> {
  typedef float type;
  __device__ static float load(float v) { return v; }
  __device__ static float store(float v) { return v; }
};
template <>
struct Elem<TF_DT_F16> {
  typedef uint16_t type;
  __device__ static float load(uint16_t v) { return f16_bits_to_f32(v); }
  __device__ static uint16_t store(float v) { return f32_to_f16_bits(v); }
};
template <>
struct Elem<TF_DT_BF16> {
  typedef uint16_t type;
  __device__ static float load(uint16_t v) { return bf16_bits_to_f32(v); }
  __device__ static uint16_t store(float v) { return f32_to_bf16_bits(v); }
};

__device__ __forceinline__ float load_elem(const void* p, int dtype, int64_t i) {
  if (dtype == TF_DT_F32) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return dtype == TF_DT_F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
}

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
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
