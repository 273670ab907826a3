// Norm of each head's query and key row and its rotation by the token's position, one pass.
//
// A workgroup takes some tokens with all their heads. The angles' cosines and sines are the
// same for every head of a token: the threads work them out once, in 64 bits up to the part of a turn,
// and leave them in shared memory. Then LANES lanes take a row, two pieces of 8 elements each, chosen
// so that both elements of every pair are in one lane: the squares' sum is LANES - 1 register moves, the
// rotation none. Bound by the rows' bytes, read once and written once.
#include <math.h>

#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

constexpr int kRotateThreads = 256;
constexpr int kTurns = 256;     // angles of a workgroup: rotary_dim / 2 a token
constexpr int kMostTokens = 8;  // of a workgroup

struct RotatePlan {
  int tokens;  // of a workgroup
  FastDiv by_rows, by_tokens, by_angles;
};

__device__ __forceinline__ void load_weights(const void* w, int dtype, int at, float (&x)[8]) {
  if (dtype == TF_DT_F32)
    load8<TF_DT_F32>(static_cast<const float*>(w) + at, x);
  else if (dtype == TF_DT_F16)
    load8<TF_DT_F16>(static_cast<const uint16_t*>(w) + at, x);
  else
    load8<TF_DT_BF16>(static_cast<const uint16_t*>(w) + at, x);
}

// Sum over aligned groups of LANES lanes, the same in each of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp<0xB1, 0xF>(v, 0.f);                           // lanes 1 apart
  v += dpp<0x4E, 0xF>(v, 0.f);                           // 2 apart
  if constexpr (LANES >= 8) v += dpp<0x141, 0xF>(v, 0.f);   // mirrored in 8: the other four
  if constexpr (LANES >= 16) v += dpp<0x140, 0xF>(v, 0.f);  // mirrored in 16: the other eight
  if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
  return v;
}

template <int DT, int LANES>
__global__ __launch_bounds__(kRotateThreads) void norm_rotate_kernel(tf_exl3_norm_rotate_args a, RotatePlan p) {
  typedef typename Elem<DT>::type T;
  __shared__ float cosines[kTurns], sines[kTurns];
  const int all = a.batch * a.tokens, first = blockIdx.x * p.tokens;
  const int here = min(p.tokens, all - first), angles = a.rotary_dim / 2;
  for (int i = threadIdx.x; i < here * angles; i += kRotateThreads) {
    const int j = p.by_angles.div(i), t = first + j, b = p.by_tokens.div(t);
    const double pos = a.positions[b * a.positions_stride + (t - b * a.tokens)];
    const double turns = pos * (double)a.frequencies[i - j * angles] * 0.15915494309189535;
    const float part = (float)(turns - rint(turns));  // within half a turn
    float s, c;
    sincospif(2.f * part, &s, &c);
    cosines[i] = c, sines[i] = s;
  }
  __syncthreads();
  const int u = threadIdx.x % LANES, rotated = a.rotary_dim / 16;
  const bool have = u < a.head_dim / 16;  // the others add zeros to the sum
  const bool turned = u < rotated;
  const bool halves = turned && !a.interleaved;
  const int at0 = halves ? 8 * u : 16 * u, at1 = halves ? angles + 8 * u : 16 * u + 8;
  const int heads = a.q_heads + a.kv_heads;
  for (int r = threadIdx.x / LANES; r < here * heads; r += kRotateThreads / LANES) {
    const int j = p.by_rows.div(r), t = first + j, b = p.by_tokens.div(t), i = t - b * a.tokens;
    const int row = r - j * heads;
    const bool query = row < a.q_heads;
    const int head = query ? row : row - a.q_heads;
    const int64_t* si = query ? a.q_stride : a.k_stride;
    const int64_t* so = query ? a.q_out_stride : a.k_out_stride;
    const T* in = static_cast<const T*>(query ? a.q : a.k) + b * si[0] + i * si[1] + head * si[2];
    T* out = static_cast<T*>(query ? a.q_out : a.k_out) + b * so[0] + i * so[1] + head * so[2];
    float x[8] = {}, y[8] = {};
    if (have) {
      load8<DT>(in + at0, x);
      load8<DT>(in + at1, y);
    }
    if (a.norm) {
      float squares = 0.f;
#pragma unroll
      for (int n = 0; n < 8; ++n) squares = __builtin_fmaf(x[n], x[n], __builtin_fmaf(y[n], y[n], squares));
      squares = lanes_sum<LANES>(squares);
      const float scale = 1.f / sqrtf(squares / (float)a.head_dim + a.eps);
      const void* w = query ? a.q_weight : a.k_weight;
#pragma unroll
      for (int n = 0; n < 8; ++n) x[n] *= scale, y[n] *= scale;
      if (w && have) {
        float w0[8], w1[8];
        load_weights(w, a.weight_dtype, at0, w0);
        load_weights(w, a.weight_dtype, at1, w1);
#pragma unroll
        for (int n = 0; n < 8; ++n) x[n] *= w0[n], y[n] *= w1[n];
      }
    }
    if (turned) {
      const float *c = cosines + j * angles + 8 * u, *s = sines + j * angles + 8 * u;
      if (a.interleaved) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float x1 = x[2 * n], x2 = x[2 * n + 1], y1 = y[2 * n], y2 = y[2 * n + 1];
          x[2 * n] = __builtin_fmaf(x1, c[n], -(x2 * s[n])), x[2 * n + 1] = __builtin_fmaf(x1, s[n], x2 * c[n]);
          y[2 * n] = __builtin_fmaf(y1, c[4 + n], -(y2 * s[4 + n]));
          y[2 * n + 1] = __builtin_fmaf(y1, s[4 + n], y2 * c[4 + n]);
        }
      } else {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float one = x[n], two = y[n];
          x[n] = __builtin_fmaf(one, c[n], -(two * s[n])), y[n] = __builtin_fmaf(one, s[n], two * c[n]);
        }
      }
    }
    if (have) {
      store8<DT>(out + at0, x);
      store8<DT>(out + at1, y);
    }
  }
}

static RotatePlan plan_of(const tf_exl3_norm_rotate_args& a) {
  const int angles = a.rotary_dim / 2 > 0 ? a.rotary_dim / 2 : 1;
  RotatePlan p;
  const int64_t share = (int64_t)a.batch * a.tokens / 1024;  // tokens of one of 1024 workgroups
  const int most = kTurns / angles < kMostTokens ? kTurns / angles : kMostTokens;
  p.tokens = share < 1 ? 1 : share < most ? (int)share : most;
  p.by_rows = fast_div(a.q_heads + a.kv_heads), p.by_tokens = fast_div(a.tokens), p.by_angles = fast_div(angles);
  return p;
}

template <int DT>
static void launch(const tf_exl3_norm_rotate_args& a, hipStream_t stream) {
  const RotatePlan p = plan_of(a);
  const dim3 grid((unsigned)(((int64_t)a.batch * a.tokens + p.tokens - 1) / p.tokens)), threads(kRotateThreads);
  if (a.head_dim <= 64)
    hipLaunchKernelGGL((norm_rotate_kernel<DT, 4>), grid, threads, 0, stream, a, p);
  else if (a.head_dim <= 128)
    hipLaunchKernelGGL((norm_rotate_kernel<DT, 8>), grid, threads, 0, stream, a, p);
  else if (a.head_dim <= 256)
    hipLaunchKernelGGL((norm_rotate_kernel<DT, 16>), grid, threads, 0, stream, a, p);
  else
    hipLaunchKernelGGL((norm_rotate_kernel<DT, 32>), grid, threads, 0, stream, a, p);
}

hipError_t launch_norm_rotate(const tf_exl3_norm_rotate_args& a, hipStream_t stream) {
  if (a.dtype == TF_DT_F32)
    launch<TF_DT_F32>(a, stream);
  else if (a.dtype == TF_DT_F16)
    launch<TF_DT_F16>(a, stream);
  else
    launch<TF_DT_BF16>(a, stream);
  return hipGetLastError();
}

}  // namespace tf_exl3
