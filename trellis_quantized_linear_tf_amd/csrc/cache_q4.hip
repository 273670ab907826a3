// Rows of keys and values into a paged cache in 4 bits, and back.
//
// Append: two lanes take a group of 32 numbers, 16 each, and minimum and maximum are one register move away. It
// takes 16 vector instructions a number, three quarters of the time that the bytes take: numbers are looked at one by
// one for what is not finite or too large only in lanes that have some, quotients are one product with a reciprocal and
// one step that rounds it as a division would, and four codes are put together as digits of one fp32 sum. 4 x 8192
// tokens of 8 heads of 128, bf16, 176 MB: 37 us, 4.8 TB/s, a copy's rate on the same card (with 8 numbers a lane and
// none of that 51 us, 28 instructions a number).
// Read: a lane takes a word of 8 codes and writes their 16 bytes; bound by them: 8 x 16384 of the same, 699 MB, in 144
// us, 4.9 TB/s.
// As many units of either are on their way a thread as hold 32 numbers.
#include "q4_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

constexpr int kQ4Threads = 256;
constexpr int kInFlight = 32;     // numbers of a thread
constexpr int kAppendUnit = 16, kReadUnit = 8;  // numbers that a thread takes at once
constexpr int kQ4MaxTokens = 64;  // tokens of a workgroup

struct Q4Plan {
  int tokens;     // of a workgroup
  int units;      // of one token: 2 heads dim / a unit's numbers
  int row_units;  // of one head's row
  FastDiv by_units, by_row, by_heads, by_page;
};

// Offsets of a token's rows: in elements outside the cache, in bytes within; k -1 where there is none.
struct Q4Row {
  int64_t k, v, k_cache, v_cache;
};

// Where position `pos` of sequence b lies in the cache, if it does.
template <typename ARGS>
__device__ __forceinline__ bool cache_place(const ARGS& a, const FastDiv& by_page, int b, int64_t pos, Q4Row* r) {
  if (pos < 0 || pos >= (int64_t)a.table_pages * a.page_size) return false;
  const int col = by_page.div((int)pos);
  const int page = a.table[b * a.table_stride + col];
  if (page < 0 || page >= a.pages) return false;
  const int slot = (int)pos - col * a.page_size;
  r->k_cache = page * a.k_cache_stride[0] + slot * a.k_cache_stride[1];
  r->v_cache = page * a.v_cache_stride[0] + slot * a.v_cache_stride[1];
  return true;
}

// Unit f of a workgroup's tokens: which token, of k (0) or v, head, and part of its row.
struct Q4Unit {
  int token, which, head, unit;
};
__device__ __forceinline__ Q4Unit unit_at(const Q4Plan& p, int heads, int f) {
  Q4Unit u;
  u.token = p.by_units.div(f);
  const int rest = f - u.token * p.units, row = p.by_row.div(rest);
  u.unit = rest - row * p.row_units;
  u.which = p.by_heads.div(row), u.head = row - u.which * heads;
  return u;
}

// Of two neighbouring lanes' numbers.
__device__ __forceinline__ float pair_min(float v) { return fminf(v, dpp<0xB1, 0xF>(v, v)); }
__device__ __forceinline__ float pair_max(float v) { return fmaxf(v, dpp<0xB1, 0xF>(v, v)); }

// d / b where that is a normal number, rounded once: `inv` is 1 / b rounded, so the product with it is off
// by an ulp at most, and its remainder, which is exact, puts it right (Markstein's theorem).
__device__ __forceinline__ float quotient(float d, float b, float inv) {
  const float t = d * inv;
  return __builtin_fmaf(__builtin_fmaf(-b, t, d), inv, t);
}

template <int DT>
__global__ __launch_bounds__(kQ4Threads) void cache_append_q4_kernel(tf_exl3_cache_append_q4_args a, Q4Plan p) {
  typedef typename Elem<DT>::type T;
  __shared__ Q4Row rows[kQ4MaxTokens];
  const int b = blockIdx.y, first = blockIdx.x * p.tokens;
  const int count = min(a.counts ? a.counts[b] : a.tokens, a.tokens);
  if (count <= first) return;
  if ((int)threadIdx.x < p.tokens) {
    Q4Row r = {-1, -1, -1, -1};
    const int j = first + threadIdx.x;
    if (j < count) {
      const int t = a.nodes ? a.nodes[(int64_t)b * a.tokens + j] : j;
      if (t >= 0 && t < a.tokens && cache_place(a, p.by_page, b, (int64_t)a.lengths[b] + j, &r)) {
        r.k = b * a.k_stride[0] + t * a.k_stride[1];
        r.v = b * a.v_stride[0] + t * a.v_stride[1];
      }
    }
    rows[threadIdx.x] = r;
  }
  __syncthreads();
  constexpr int kUnits = kInFlight / kAppendUnit, kPieces = kAppendUnit * (int)sizeof(T) / 16;
  const int all = p.tokens * p.units;
  for (int f0 = threadIdx.x; f0 < all; f0 += kQ4Threads * kUnits) {
    u32x4 raw[kUnits][kPieces];
    uint8_t* to[kUnits];  // the row in the cache
    int unit[kUnits];
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int f = f0 + n * kQ4Threads;
      to[n] = nullptr;
      if (f >= all) continue;
      const Q4Unit u = unit_at(p, a.kv_heads, f);
      const Q4Row& r = rows[u.token];
      if (r.k < 0) continue;
      unit[n] = u.unit;
      const T* from = u.which ? static_cast<const T*>(a.v) + r.v + u.head * a.v_stride[2]
                              : static_cast<const T*>(a.k) + r.k + u.head * a.k_stride[2];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) raw[n][i] = load_piece(from + kAppendUnit * u.unit + i * (16 / (int)sizeof(T)));
      to[n] = u.which ? static_cast<uint8_t*>(a.v_cache) + r.v_cache + u.head * a.v_cache_stride[2]
                      : static_cast<uint8_t*>(a.k_cache) + r.k_cache + u.head * a.k_cache_stride[2];
    }
    // The two lanes of a group are here together or not at all: a row has whole groups.
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      if (!to[n]) continue;
      float x[kAppendUnit];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        constexpr int kEach = 16 / (int)sizeof(T);
        float y[kEach];
        Elem<DT>::unpack(raw[n][i], y);
#pragma unroll
        for (int j = 0; j < kEach; ++j) x[i * kEach + j] = y[j];
      }
      float low = x[0], high = x[0], odd = 0.f;  // odd: NaN where a number is not finite
#pragma unroll
      for (int i = 0; i < kAppendUnit; ++i) {
        low = fminf(low, x[i]), high = fmaxf(high, x[i]);
        odd = __builtin_fmaf(x[i], 0.f, odd);
      }
      if (!(odd == 0.f && low >= -kQ4Most && high <= kQ4Most)) {
        low = INFINITY, high = -INFINITY;
#pragma unroll
        for (int i = 0; i < kAppendUnit; ++i) {
          const float v = x[i] == x[i] ? x[i] : 0.f;
          x[i] = fminf(fmaxf(v, -kQ4Most), kQ4Most);
          low = fminf(low, x[i]), high = fmaxf(high, x[i]);
        }
      }
      low = pair_min(low), high = pair_max(high);
      // Rounded to fp32 first, where a mixed multiply-add would round to fp16 alone.
      const uint16_t scale_bits = f32_to_f16_bits(opaque(quotient(high - low, 15.f, 1.f / 15.f)));
      uint16_t low_bits = f32_to_f16_bits(low);
      if (low_bits == 0x8000u) low_bits = 0;  // of zeros of both signs either may be the smallest
      const float scale = f16_bits_to_f32(scale_bits), from = f16_bits_to_f32(low_bits);
      // 1 / scale rounded: one step of Newton's from within an ulp (exact but for significands of ones only,
      // which 11 bits are not).
      float inv = __builtin_amdgcn_rcpf(scale);
      inv = scale > 0.f ? __builtin_fmaf(__builtin_fmaf(-scale, inv, 1.f), inv, inv) : 0.f;
      uint32_t word[kAppendUnit / 8];
#pragma unroll
      for (int w = 0; w < kAppendUnit / 8; ++w) {
        float code[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)  // rounded as a division would be where it is not 0 or 15 anyway
          code[i] = __builtin_amdgcn_fmed3f(rintf(quotient(x[8 * w + i] - from, scale, inv)), 0.f, 15.f);
        float halves[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          halves[h] = code[6 + h];
#pragma unroll
          for (int i = 2; i >= 0; --i) halves[h] = __builtin_fmaf(halves[h], 16.f, code[2 * i + h]);
        }
        word[w] = (uint32_t)halves[1] << 16 | (uint32_t)halves[0];
      }
      typedef uint32_t words __attribute__((ext_vector_type(2), aligned(4)));
      reinterpret_cast<words*>(to[n])[unit[n]] = words{word[0], word[1]};
      if ((unit[n] & 1) == 0)
        reinterpret_cast<uint32_t*>(to[n] + a.head_dim / 2)[unit[n] >> 1] = (uint32_t)low_bits << 16 | scale_bits;
    }
  }
}

template <int DT>
__global__ __launch_bounds__(kQ4Threads) void cache_read_q4_kernel(tf_exl3_cache_read_q4_args a, Q4Plan p) {
  typedef typename Elem<DT>::type T;
  __shared__ Q4Row rows[kQ4MaxTokens];
  const int b = blockIdx.y, first = blockIdx.x * p.tokens;
  if ((int)threadIdx.x < p.tokens) {
    Q4Row r = {-1, -1, -1, -1};
    const int j = first + threadIdx.x;
    if (j < a.tokens) {
      const int64_t pos = (a.first ? (int64_t)a.first[b] : 0) + j;
      if (pos >= a.lengths[b] || !cache_place(a, p.by_page, b, pos, &r)) r.k_cache = -1;
      r.k = b * a.k_stride[0] + j * a.k_stride[1];
      r.v = b * a.v_stride[0] + j * a.v_stride[1];
    }
    rows[threadIdx.x] = r;
  }
  __syncthreads();
  constexpr int kUnits = kInFlight / kReadUnit;
  const int all = p.tokens * p.units;
  for (int f0 = threadIdx.x; f0 < all; f0 += kQ4Threads * kUnits) {
    uint32_t word[kUnits], pair[kUnits];
    T* to[kUnits];
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      const int f = f0 + n * kQ4Threads;
      to[n] = nullptr, word[n] = pair[n] = 0;
      if (f >= all) continue;
      const Q4Unit u = unit_at(p, a.kv_heads, f);
      const Q4Row& r = rows[u.token];
      if (r.k < 0) continue;
      const uint8_t* from;
      if (u.which) {
        to[n] = static_cast<T*>(a.v) + r.v + u.head * a.v_stride[2] + kReadUnit * u.unit;
        from = static_cast<const uint8_t*>(a.v_cache) + r.v_cache + u.head * a.v_cache_stride[2];
      } else {
        to[n] = static_cast<T*>(a.k) + r.k + u.head * a.k_stride[2] + kReadUnit * u.unit;
        from = static_cast<const uint8_t*>(a.k_cache) + r.k_cache + u.head * a.k_cache_stride[2];
      }
      if (r.k_cache < 0) continue;  // codes, scale and minimum of 0 are zeros
      word[n] = reinterpret_cast<const uint32_t*>(from)[u.unit];
      pair[n] = reinterpret_cast<const uint32_t*>(from + a.head_dim / 2)[u.unit >> 2];
    }
#pragma unroll
    for (int n = 0; n < kUnits; ++n) {
      if (!to[n]) continue;
      if constexpr (DT == TF_DT_F32) {
        float x[8];
        q4_values(word[n], q4_unpack(pair[n]), x);
        store8<DT>(to[n], x);
      } else {
        store_piece(to[n], q4_piece<DT>(word[n], pair[n]));
      }
    }
  }
}

template <typename ARGS>
static Q4Plan plan_of(const ARGS& a, int unit) {
  Q4Plan p;
  p.row_units = a.head_dim / unit;
  p.units = 2 * a.kv_heads * p.row_units;
  // Up to as many tokens as one round of the threads' numbers holds, but first 1024 workgroups, four a CU. 1, 2, 4
  // tokens, us on the GPU, 8 heads of 128: append and read of 4 x 64 tokens 6.2 / 6.5 / 7.9, of 4 x 1024 18.3 / 15.4 /
  // 15.2; read of 8 x 16384 224 / 162 / 149.
  const int round = kQ4Threads * (kInFlight / unit) / p.units;
  const int most = round < 1 ? 1 : round < kQ4MaxTokens ? round : kQ4MaxTokens;
  const int64_t share = (int64_t)a.batch * a.tokens / 1024;
  p.tokens = share < 1 ? 1 : share < most ? (int)share : most;
  p.by_units = fast_div(p.units), p.by_row = fast_div(p.row_units);
  p.by_heads = fast_div(a.kv_heads), p.by_page = fast_div(a.page_size);
  return p;
}

template <typename ARGS>
static dim3 grid_of(const ARGS& a, const Q4Plan& p) {
  return dim3((unsigned)(((int64_t)a.tokens + p.tokens - 1) / p.tokens), a.batch);
}

bool cache_append_q4_fits(const tf_exl3_cache_append_q4_args& a) {
  return launchable(grid_of(a, plan_of(a, kAppendUnit)).x, kQ4Threads);
}
bool cache_read_q4_fits(const tf_exl3_cache_read_q4_args& a) {
  return launchable(grid_of(a, plan_of(a, kReadUnit)).x, kQ4Threads);
}

hipError_t launch_cache_append_q4(const tf_exl3_cache_append_q4_args& a, hipStream_t stream) {
  const Q4Plan p = plan_of(a, kAppendUnit);
  const dim3 grid = grid_of(a, p), threads(kQ4Threads);
  if (a.dtype == TF_DT_F32)
    hipLaunchKernelGGL(cache_append_q4_kernel<TF_DT_F32>, grid, threads, 0, stream, a, p);
  else if (a.dtype == TF_DT_F16)
    hipLaunchKernelGGL(cache_append_q4_kernel<TF_DT_F16>, grid, threads, 0, stream, a, p);
  else
    hipLaunchKernelGGL(cache_append_q4_kernel<TF_DT_BF16>, grid, threads, 0, stream, a, p);
  return hipGetLastError();
}

hipError_t launch_cache_read_q4(const tf_exl3_cache_read_q4_args& a, hipStream_t stream) {
  const Q4Plan p = plan_of(a, kReadUnit);
  const dim3 grid = grid_of(a, p), threads(kQ4Threads);
  if (a.dtype == TF_DT_F32)
    hipLaunchKernelGGL(cache_read_q4_kernel<TF_DT_F32>, grid, threads, 0, stream, a, p);
  else if (a.dtype == TF_DT_F16)
    hipLaunchKernelGGL(cache_read_q4_kernel<TF_DT_F16>, grid, threads, 0, stream, a, p);
  else
    hipLaunchKernelGGL(cache_read_q4_kernel<TF_DT_BF16>, grid, threads, 0, stream, a, p);
  return hipGetLastError();
}

}  // namespace tf_exl3
