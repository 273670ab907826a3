// Norm of each head's query and key row and its rotation by the token's position, one pass.
//
// A workgroup takes some tokens with all their heads. The angles' cosines and sines are the
// same for every head of a token: the threads work them out once, in 64 bits up to the part of a turn,
// and leave them in shared memory. Then LANES lanes take a row, two pieces of 8 elements each, chosen
// so that both elements of every pair are in one lane: the squares' sum is log2(LANES) register moves, the
// rotation none. Bound by the rows' bytes, read once and written once: a row is on its way while the one before is
// worked at, the first of them while the angles are. 4 x 4099 tokens of 40 rows of 128, bf16, 336 MB: 74 us, 4.5 TB/s,
// where a copy of 4 GiB reached 4.7 on the same card.
#include <math.h>

#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

constexpr int kRotateThreads = 256;
constexpr int kTurns = 256;     // angles of a workgroup: rotary_dim / 2 a token
constexpr int kMostTokens = 8;  // of a workgroup

struct RotatePlan {
  int tokens;  // of a workgroup
  int parts;   // workgroups that share its rows
  FastDiv by_q_heads, by_kv_heads, by_tokens, by_angles;
};

typedef uint32_t u32x2_elem __attribute__((ext_vector_type(2), aligned(2)));

// Two pieces of eight elements of a row, as they lie there.
template <int DT>
struct RawRow {
  static constexpr int kPieces = DT == TF_DT_F32 ? 2 : 1;
  u32x4 x[kPieces], y[kPieces];
};

template <int DT>
__device__ __forceinline__ void numbers(const u32x4 (&raw)[RawRow<DT>::kPieces], float (&x)[8]) {
  if constexpr (DT == TF_DT_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bits_to_f32(raw[i / 4][i % 4]);
  } else {
    Elem<DT>::unpack(raw[0], x);
  }
}

// The same of a row whose last pair of turned pieces is half of each: elements 4 to 7 of a piece stand elsewhere.
template <int DT>
__device__ __forceinline__ void load_halves(const typename Elem<DT>::type* first, const typename Elem<DT>::type* last,
                                            u32x4 (&raw)[RawRow<DT>::kPieces]) {
  if constexpr (DT == TF_DT_F32) {
    raw[0] = load_piece(first), raw[1] = load_piece(last);
  } else {
    const u32x2_elem a = *reinterpret_cast<const u32x2_elem*>(first), b = *reinterpret_cast<const u32x2_elem*>(last);
    raw[0] = u32x4{a[0], a[1], b[0], b[1]};
  }
}
template <int DT>
__device__ __forceinline__ void store_halves(typename Elem<DT>::type* first, typename Elem<DT>::type* last, const float (&x)[8]) {
  if constexpr (DT == TF_DT_F32) {
    store_piece(first, u32x4{f32_to_bits(x[0]), f32_to_bits(x[1]), f32_to_bits(x[2]), f32_to_bits(x[3])});
    store_piece(last, u32x4{f32_to_bits(x[4]), f32_to_bits(x[5]), f32_to_bits(x[6]), f32_to_bits(x[7])});
  } else {
    const u32x4 v = Elem<DT>::pack(x);
    *reinterpret_cast<u32x2_elem*>(first) = u32x2_elem{v[0], v[1]};
    *reinterpret_cast<u32x2_elem*>(last) = u32x2_elem{v[2], v[3]};
  }
}

__device__ __forceinline__ void load_weights(const void* w, int dtype, int at, float (&x)[8]) {
  if (dtype == TF_DT_F32)
    load8<TF_DT_F32>(static_cast<const float*>(w) + at, x);
  else if (dtype == TF_DT_F16)
    load8<TF_DT_F16>(static_cast<const uint16_t*>(w) + at, x);
  else
    load8<TF_DT_BF16>(static_cast<const uint16_t*>(w) + at, x);
}

// f over aligned groups of LANES lanes, the same in each of them.
template <int LANES, typename F>
__device__ __forceinline__ float lanes_join(float v, F f) {
  v = f(v, dpp<0xB1, 0xF>(v, 0.f));                           // lanes 1 apart
  v = f(v, dpp<0x4E, 0xF>(v, 0.f));                           // 2 apart
  if constexpr (LANES >= 8) v = f(v, dpp<0x141, 0xF>(v, 0.f));   // mirrored in 8: the other four
  if constexpr (LANES >= 16) v = f(v, dpp<0x140, 0xF>(v, 0.f));  // mirrored in 16: the other eight
  if constexpr (LANES >= 32) v = f(v, __shfl_xor(v, 16));
  return v;
}

// Mean of the row's squares.
template <int LANES>
__device__ __forceinline__ float mean_square(const float (&x)[8], const float (&y)[8], int dim) {
  float squares = 0.f;
#pragma unroll
  for (int n = 0; n < 8; ++n) squares = __builtin_fmaf(x[n], x[n], __builtin_fmaf(y[n], y[n], squares));
  return lanes_join<LANES>(squares, [](float u, float v) { return u + v; }) / (float)dim;
}

// SPLIT: rotary_dim is 8 more than a multiple of 16. The last lane that turns has half a piece of either half, and
// makes its pieces whole with what stands behind rotary_dim. Pieces go by halves then: 16384 tokens of 40 rows of 96, bf16,
// 24 turned 68 us, 32 turned 50; of 128, 120 turned 95 us, 128 turned 71.
template <int DT, int LANES, bool SPLIT>
__global__ __launch_bounds__(kRotateThreads) void norm_rotate_kernel(tf_exl3_norm_rotate_args a, RotatePlan p) {
  typedef typename Elem<DT>::type T;
  __shared__ float cosines[kTurns], sines[kTurns];
  const int all = a.batch * a.tokens, first = blockIdx.x * p.tokens;
  const int here = min(p.tokens, all - first), angles = a.rotary_dim / 2;
  const int u = threadIdx.x % LANES;
  const bool have = u < a.head_dim / 16;  // the others add zeros to the sum
  const bool turned = 16 * u < a.rotary_dim;
  const bool all_turned = !SPLIT || 16 * u + 8 < a.rotary_dim;  // not only the first halves of its pieces' pairs
  const bool halves = turned && !a.interleaved;
  const int at0 = halves ? 8 * u : 16 * u, at1 = halves ? angles + 8 * u : 16 * u + 8;
  const bool apart = halves && !all_turned;
  const int rest0 = apart ? a.rotary_dim : at0 + 4, rest1 = apart ? a.rotary_dim + 4 : at1 + 4;

  // Rows in this order: the tokens' queries, then their keys.
  struct Place {
    const T* in;
    T* out;
    int token;  // of the workgroup's
    bool query;
  };
  const int queries = here * a.q_heads, rows = queries + here * a.kv_heads;
  auto place = [&](int r) {
    Place x;
    x.query = r < queries;
    const int row = x.query ? r : r - queries;
    x.token = (x.query ? p.by_q_heads : p.by_kv_heads).div(row);
    const int head = row - x.token * (x.query ? a.q_heads : a.kv_heads);
    const int t = first + x.token, b = p.by_tokens.div(t), i = t - b * a.tokens;
    const int64_t* si = x.query ? a.q_stride : a.k_stride;
    const int64_t* so = x.query ? a.q_out_stride : a.k_out_stride;
    auto offset = [&](const int64_t* s) {  // below 2^32 each
      return (uint64_t)(uint32_t)b * (uint32_t)s[0] + (uint64_t)(uint32_t)i * (uint32_t)s[1] + (uint64_t)(uint32_t)head * (uint32_t)s[2];
    };
    x.in = static_cast<const T*>(x.query ? a.q : a.k) + offset(si);
    x.out = static_cast<T*>(x.query ? a.q_out : a.k_out) + offset(so);
    return x;
  };
  auto load = [&](const Place& x, RawRow<DT>& raw) {
    if constexpr (SPLIT) {
#pragma unroll
      for (int n = 0; n < RawRow<DT>::kPieces; ++n) raw.x[n] = raw.y[n] = u32x4(0u);
      if (have) {
        load_halves<DT>(x.in + at0, x.in + rest0, raw.x);
        load_halves<DT>(x.in + at1, x.in + rest1, raw.y);
      }
      return;
    }
#pragma unroll
    for (int n = 0; n < RawRow<DT>::kPieces; ++n) {
      raw.x[n] = raw.y[n] = u32x4(0u);
      if (have) raw.x[n] = load_piece(x.in + at0 + 4 * n), raw.y[n] = load_piece(x.in + at1 + 4 * n);
    }
  };

  constexpr int kSlots = kRotateThreads / LANES;
  const int step = kSlots * p.parts;
  int r = blockIdx.y * kSlots + threadIdx.x / LANES;
  Place now = {};
  RawRow<DT> raw = {};
  if (r < rows) {
    now = place(r);
    load(now, raw);
  }
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

  float w0[8], w1[8];
  int weights_of = -1;  // keys (0) or queries
  while (r < rows) {
    const int ahead = r + step;
    Place next = {};
    RawRow<DT> raw_next = {};
    if (ahead < rows) {
      next = place(ahead);
      load(next, raw_next);
    }
    float x[8], y[8];
    numbers<DT>(raw.x, x);
    numbers<DT>(raw.y, y);
    if (a.norm) {
      if (weights_of != (int)now.query) {
        weights_of = now.query;
        const void* w = now.query ? a.q_weight : a.k_weight;
#pragma unroll
        for (int n = 0; n < 8; ++n) w0[n] = w1[n] = 1.f;
        if (w && have) {
          if constexpr (SPLIT) {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              w0[n] = load_elem(w, a.weight_dtype, (n < 4 ? at0 : rest0 - 4) + n);
              w1[n] = load_elem(w, a.weight_dtype, (n < 4 ? at1 : rest1 - 4) + n);
            }
          } else {
            load_weights(w, a.weight_dtype, at0, w0);
            load_weights(w, a.weight_dtype, at1, w1);
          }
        }
      }
      float square = mean_square<LANES>(x, y, a.head_dim) + a.eps;
      // Squares near the ends of fp32: the row, and the square root of eps, in units of a power of two in which the largest
      // of them is about 1. All of a row's lanes come here together. (Squares of fp16 are far from them.)
      if (DT != TF_DT_F16 && !(square > 0x1p-80f && square < 0x1p120f)) {
        float most = sqrtf(a.eps);
#pragma unroll
        for (int n = 0; n < 8; ++n) most = fmaxf(most, fmaxf(fabsf(x[n]), fabsf(y[n])));
        most = lanes_join<LANES>(most, [](float u, float v) { return fmaxf(u, v); });
        // 0 for 0 and infinity, whose rows stay what they are
        const float unit = ldexpf(1.f, min(max(-__builtin_amdgcn_frexp_expf(most), -126), 126));
#pragma unroll
        for (int n = 0; n < 8; ++n) x[n] *= unit, y[n] *= unit;
        square = mean_square<LANES>(x, y, a.head_dim) + a.eps * unit * unit;
      }
      const float scale = 1.f / sqrtf(square);
#pragma unroll
      for (int n = 0; n < 8; ++n) x[n] = x[n] * scale * w0[n], y[n] = y[n] * scale * w1[n];
    }
    if (turned) {
      const float *c = cosines + now.token * angles + 8 * u, *s = sines + now.token * angles + 8 * u;
      if (a.interleaved) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float x1 = x[2 * n], x2 = x[2 * n + 1], y1 = y[2 * n], y2 = y[2 * n + 1];
          x[2 * n] = __builtin_fmaf(x1, c[n], -(x2 * s[n])), x[2 * n + 1] = __builtin_fmaf(x1, s[n], x2 * c[n]);
          if (!all_turned) continue;
          y[2 * n] = __builtin_fmaf(y1, c[4 + n], -(y2 * s[4 + n]));
          y[2 * n + 1] = __builtin_fmaf(y1, s[4 + n], y2 * c[4 + n]);
        }
      } else {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          if (n >= 4 && !all_turned) continue;
          const float one = x[n], two = y[n];
          x[n] = __builtin_fmaf(one, c[n], -(two * s[n])), y[n] = __builtin_fmaf(one, s[n], two * c[n]);
        }
      }
    }
    if (have) {
      if constexpr (SPLIT) {
        store_halves<DT>(now.out + at0, now.out + rest0, x);
        store_halves<DT>(now.out + at1, now.out + rest1, y);
      } else {
        store8<DT>(now.out + at0, x);
        store8<DT>(now.out + at1, y);
      }
    }
    r = ahead, now = next, raw = raw_next;
  }
}

static RotatePlan plan_of(const tf_exl3_norm_rotate_args& a, int slots) {
  const int angles = a.rotary_dim / 2 > 0 ? a.rotary_dim / 2 : 1;
  RotatePlan p;
  const int64_t all = (int64_t)a.batch * a.tokens, share = all / 1024;  // tokens of one of 1024 workgroups
  const int most = kTurns / angles < kMostTokens ? kTurns / angles : kMostTokens;
  // 1, 2, 4, 8 tokens a workgroup, us on the GPU, 40 rows of 128 a token: 1024 tokens 7.0 / 7.1 / 8.4 / 11.8, 2048
  // 11.8 / 10.5 / 10.8 / 13.7, 4096 20.0 / 18.3 / 16.4 / 17.3, 16384 89 / 75 / 71 / 71.
  p.tokens = share < 1 ? 1 : share < most ? (int)share : most;
  // Few tokens: their rows are shared out, as far as each thread still has one. One workgroup a token against that, us:
  // 1 token 4.1 / 3.3, 512 5.2 / 4.7, 1024 7.1 / 7.8, 4096 16.5 / 17.2 (5 rows of 256 a token: the same at all of them).
  const int rows = (a.q_heads + a.kv_heads + slots - 1) / slots;
  p.parts = all > 512 ? 1 : rows;
  p.by_q_heads = fast_div(a.q_heads), p.by_kv_heads = fast_div(a.kv_heads);
  p.by_tokens = fast_div(a.tokens), p.by_angles = fast_div(angles);
  return p;
}

template <int DT, int LANES>
static void launch(const tf_exl3_norm_rotate_args& a, hipStream_t stream) {
  const RotatePlan p = plan_of(a, kRotateThreads / LANES);
  const dim3 grid((unsigned)(((int64_t)a.batch * a.tokens + p.tokens - 1) / p.tokens), p.parts), threads(kRotateThreads);
  if (a.rotary_dim % 16 == 0)
    hipLaunchKernelGGL((norm_rotate_kernel<DT, LANES, false>), grid, threads, 0, stream, a, p);
  else
    hipLaunchKernelGGL((norm_rotate_kernel<DT, LANES, true>), grid, threads, 0, stream, a, p);
}

template <int DT>
static void launch(const tf_exl3_norm_rotate_args& a, hipStream_t stream) {
  if (a.head_dim <= 64)
    launch<DT, 4>(a, stream);
  else if (a.head_dim <= 128)
    launch<DT, 8>(a, stream);
  else if (a.head_dim <= 256)
    launch<DT, 16>(a, stream);
  else
    launch<DT, 32>(a, stream);
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
