// Rows of keys and values into a paged cache, byte for byte. Nothing is computed, so the
// bytes, read once and written once, are the whole cost: every thread has kCopies
// independent loads in flight before its first store. 32768 tokens of 8 heads of 128, bf16 keys
// and values into pages: 268 MB read and written in 57 us, 4.7 TB/s (element by element 107). The times at the
// rule below are of inputs that stay in the caches from pass to pass: 45 us for the same tokens.
#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

constexpr int kAppendThreads = 256;
constexpr int kCopies = 8;     // units a thread copies at a time
constexpr int kMaxTokens = 64;  // tokens of a workgroup

template <int BYTES>
struct Unit;
template <>
struct Unit<16> { typedef u32x4 type; };
template <>
struct Unit<4> { typedef uint32_t type; };
template <>
struct Unit<2> { typedef uint16_t type; };
template <>
struct Unit<1> { typedef uint8_t type; };

struct AppendPlan {
  int tokens;          // of a workgroup
  int units;           // of one token: 2 heads dim elem_bytes / BYTES
  int row_units;       // of one head's row
  FastDiv by_units, by_row, by_heads, by_page;
};

// Offsets in bytes of a token's rows, -1 where it writes nothing.
struct TokenRow {
  int64_t k, v, k_cache, v_cache;
};

__device__ __forceinline__ TokenRow token_row(const tf_exl3_cache_append_args& a, const FastDiv& by_page, int b, int j) {
  TokenRow r = {-1, -1, -1, -1};
  const int count = a.counts ? a.counts[b] : a.tokens;
  if (j >= a.tokens || j >= count) return r;
  const int t = a.nodes ? a.nodes[(int64_t)b * a.tokens + j] : j;
  const int64_t pos = (int64_t)a.lengths[b] + j;
  if (t < 0 || t >= a.tokens || pos < 0 || pos >= (int64_t)a.table_pages * a.page_size) return r;
  const int col = by_page.div((int)pos);
  const int page = a.table[b * a.table_stride + col];
  if (page < 0 || page >= a.pages) return r;
  const int slot = (int)pos - col * a.page_size, e = a.elem_bytes;
  r.k = (b * a.k_stride[0] + t * a.k_stride[1]) * e;
  r.v = (b * a.v_stride[0] + t * a.v_stride[1]) * e;
  r.k_cache = (page * a.k_cache_stride[0] + slot * a.k_cache_stride[1]) * e;
  r.v_cache = (page * a.v_cache_stride[0] + slot * a.v_cache_stride[1]) * e;
  return r;
}

// One workgroup per sequence and group of tokens. Unit f of the group is token f / units,
// then k or v, head and place in the head's row.
template <int BYTES>
__global__ __launch_bounds__(kAppendThreads) void cache_append_kernel(tf_exl3_cache_append_args a, AppendPlan p) {
  typedef typename Unit<BYTES>::type T;
  __shared__ TokenRow rows[kMaxTokens];
  const int b = blockIdx.y, first = blockIdx.x * p.tokens;
  if (a.counts && a.counts[b] <= first) return;
  if ((int)threadIdx.x < p.tokens) rows[threadIdx.x] = token_row(a, p.by_page, b, first + threadIdx.x);
  __syncthreads();
  const int all = p.tokens * p.units;
  for (int f0 = threadIdx.x; f0 < all; f0 += kAppendThreads * kCopies) {
    T data[kCopies];
    T* to[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int f = f0 + i * kAppendThreads;
      to[i] = nullptr;
      if (f < all) {
        const int token = p.by_units.div(f), rest = f - token * p.units;
        const int row = p.by_row.div(rest), unit = rest - row * p.row_units;
        const int which = p.by_heads.div(row), h = row - which * a.kv_heads;
        const TokenRow& r = rows[token];
        if (r.k >= 0) {
          const int64_t at = (int64_t)unit * BYTES;
          const char* from = which ? static_cast<const char*>(a.v) + r.v + h * a.v_stride[2] * a.elem_bytes
                                   : static_cast<const char*>(a.k) + r.k + h * a.k_stride[2] * a.elem_bytes;
          char* dst = which ? static_cast<char*>(a.v_cache) + r.v_cache + h * a.v_cache_stride[2] * a.elem_bytes
                            : static_cast<char*>(a.k_cache) + r.k_cache + h * a.k_cache_stride[2] * a.elem_bytes;
          data[i] = *reinterpret_cast<const T*>(from + at);
          to[i] = reinterpret_cast<T*>(dst + at);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kCopies; ++i)
      if (to[i]) *to[i] = data[i];
  }
}

// Whether every row begins and ends at a multiple of `bytes`.
static bool in_units(const tf_exl3_cache_append_args& a, int bytes) {
  const int e = a.elem_bytes;
  if ((a.head_dim * e) % bytes) return false;
  const void* at[4] = {a.k, a.v, a.k_cache, a.v_cache};
  const int64_t* strides[4] = {a.k_stride, a.v_stride, a.k_cache_stride, a.v_cache_stride};
  for (int i = 0; i < 4; ++i) {
    if ((uintptr_t)at[i] % bytes) return false;
    for (int j = 0; j < 3; ++j)
      if ((strides[i][j] * e) % bytes) return false;
  }
  return true;
}

template <int BYTES>
static AppendPlan plan_of(const tf_exl3_cache_append_args& a) {
  AppendPlan p;
  p.row_units = a.head_dim * a.elem_bytes / BYTES;
  p.units = 2 * a.kv_heads * p.row_units;
  // Up to as many tokens as one round of the threads' copies holds, but first 1024 workgroups.
  // One token each against a full round, us: 64 x 16 tokens of 8 heads of 128 4.0 / 5.5, 4 x 512 5.8 /
  // 6.1, 4 x 2048 15.5 / 12.2, 4 x 8192 63 / 45; 64 x 128 of one head of 64 8.6 / 4.0.
  const int round = kAppendThreads * kCopies / p.units;
  const int most = round < 1 ? 1 : round < kMaxTokens ? round : kMaxTokens;
  const int64_t share = (int64_t)a.batch * a.tokens / 1024;
  p.tokens = share < 1 ? 1 : share < most ? (int)share : most;
  p.by_units = fast_div(p.units), p.by_row = fast_div(p.row_units);
  p.by_heads = fast_div(a.kv_heads), p.by_page = fast_div(a.page_size);
  return p;
}

static int unit_of(const tf_exl3_cache_append_args& a) { return in_units(a, 16) ? 16 : in_units(a, 4) ? 4 : in_units(a, 2) ? 2 : 1; }

static AppendPlan plan_of(const tf_exl3_cache_append_args& a, int unit) {
  return unit == 16 ? plan_of<16>(a) : unit == 4 ? plan_of<4>(a) : unit == 2 ? plan_of<2>(a) : plan_of<1>(a);
}

static int64_t workgroups_of(const tf_exl3_cache_append_args& a, const AppendPlan& p) {
  return ((int64_t)a.tokens + p.tokens - 1) / p.tokens;
}

template <int BYTES>
static void launch(const tf_exl3_cache_append_args& a, const AppendPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL(cache_append_kernel<BYTES>, dim3((unsigned)workgroups_of(a, p), a.batch), dim3(kAppendThreads), 0,
                     stream, a, p);
}

bool cache_append_fits(const tf_exl3_cache_append_args& a) {
  return launchable(workgroups_of(a, plan_of(a, unit_of(a))), kAppendThreads);
}

hipError_t launch_cache_append(const tf_exl3_cache_append_args& a, hipStream_t stream) {
  const int unit = unit_of(a);
  const AppendPlan p = plan_of(a, unit);
  if (unit == 16)
    launch<16>(a, p, stream);
  else if (unit == 4)
    launch<4>(a, p, stream);
  else if (unit == 2)
    launch<2>(a, p, stream);
  else
    launch<1>(a, p, stream);
  return hipGetLastError();
}

}  // namespace tf_exl3
