// Distillation from a teacher's top logits: the loss of each row and its gradient.
//
// With d = x - max x, the student's p[i] = 2^(d c) / z, c = log2(e) / T, z their sum; a
// row's loss and gradient need z and the maximum before anything can be written, so a
// row is read, held on chip where it fits, and the gradient written from what is held.
#include <math.h>

#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

constexpr int kMaxTop = 1024;

// 2^(d c) with c in two parts: the product's error is then one rounding of the
// exponent and not the rounding of c times |d|, which all elements would share.
struct Scale {
  float inv, c, c_low;
  __device__ float exp(float d) const {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(d, c, d * c_low));
  }
};

__device__ __forceinline__ Scale scale_of(float temperature) {
  Scale s;
  const double c = 1.4426950408889634 / (double)temperature;
  s.inv = 1.f / temperature;
  s.c = (float)c;
  s.c_low = (float)(c - (double)s.c);
  return s;
}

template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N], float m) {
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, x[i]);
  return m;
}

// Sum of a thread's accumulators, in pairs.
template <int N>
__device__ __forceinline__ float sum_of(float (&s)[N]) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) s[i] += s[i + o];
  return s[0];
}

struct Teacher {
  float t[kMaxTop];  // logit, then probability
  int at[kMaxTop];   // place, -1 for an entry that is left out
};

// The teacher's entries into shared memory.
template <int THREADS>
__device__ __forceinline__ void load_teacher(const DistillArgs& a, int64_t r, Teacher& s) {
  for (int j = threadIdx.x; j < a.top_k; j += THREADS) {
    const int i = a.index[r * a.top_k + j];
    const bool there = i >= 0 && i < a.vocab;
    s.at[j] = there ? i : -1;
    s.t[j] = there ? load_elem(a.top, a.top_dtype, r * a.top_k + j) : -INFINITY;
  }
}

// Its probabilities and the row's loss, given the student's maximum and sum. Each thread
// meets only entries of its own until the barrier inside the last sum.
template <int THREADS, int DT>
__device__ __forceinline__ float teacher_loss(const DistillArgs& a, const Scale& sc, const typename Elem<DT>::type* x,
                                              float top, float z, Teacher& s, float* red, bool* none) {
  constexpr int kWaves = THREADS / 64;
  float ymax = -INFINITY;
  for (int j = threadIdx.x; j < a.top_k; j += THREADS) ymax = fmaxf(ymax, s.t[j]);
  ymax = block_max<kWaves>(ymax, red);
  float ysum = 0.f;
  for (int j = threadIdx.x; j < a.top_k; j += THREADS) ysum += s.at[j] >= 0 ? sc.exp(s.t[j] - ymax) : 0.f;
  ysum = block_sum<kWaves>(ysum, red);
  *none = ysum == 0.f;
  const float lz = logf(z), lys = logf(ysum);
  float loss = 0.f;
  for (int j = threadIdx.x; j < a.top_k; j += THREADS) {
    float t = 0.f;
    if (s.at[j] >= 0) {
      const float ly = (s.t[j] - ymax) * sc.inv - lys;
      t = sc.exp(s.t[j] - ymax) / ysum;
      if (t > 0.f) loss += t * (ly - ((Elem<DT>::load(x[s.at[j]]) - top) * sc.inv - lz));
    }
    s.t[j] = t;
  }
  return block_sum<kWaves>(loss, red);
}

// The gradient at the teacher's places within [lo, hi), over what the row's pieces left
// there. The first of equal places holds the sum of them all, in order.
template <int THREADS, int DT>
__device__ __forceinline__ void teacher_grad(const DistillArgs& a, const Scale& sc, const typename Elem<DT>::type* x,
                                             typename Elem<DT>::type* grad, float top, float z, float w, const Teacher& s,
                                             int lo, int hi) {
  for (int j = threadIdx.x; j < a.top_k; j += THREADS) {
    const int at = s.at[j];
    if (at < lo || at >= hi) continue;
    float t = 0.f;
    bool first = true;
    for (int i = 0; i < a.top_k; ++i)
      if (s.at[i] == at) {
        first = first && i >= j;
        t += s.t[i];
      }
    if (first) grad[at] = Elem<DT>::store((sc.exp(Elem<DT>::load(x[at]) - top) / z - t) * w);
  }
}

template <int DT>
__device__ __forceinline__ u32x4 grad_piece(u32x4 v, const Scale& sc, float top, float w_z, bool zero) {
  constexpr int P = Elem<DT>::kPiece;
  if (zero) return u32x4(0u);  // whatever the row holds
  float e[P];
  Elem<DT>::unpack(v, e);
#pragma unroll
  for (int i = 0; i < P; ++i) e[i] = sc.exp(e[i] - top) * w_z;
  return Elem<DT>::pack(e);
}

// One workgroup per row, N pieces of 16 bytes held by each thread; what a longer row has
// beyond them is read first, with a running maximum, and once more for the gradient
// (then from the memory-side cache: the rows in flight are below its 256 MB). The
// sums' order depends on the row's length alone, so the loss has the same bits with and
// without the gradient.
template <int DT, int THREADS, int N>
__global__ __launch_bounds__(THREADS) void distill_row_kernel(DistillArgs a) {
  typedef typename Elem<DT>::type T;
  constexpr int P = Elem<DT>::kPiece, kWaves = THREADS / 64;
  __shared__ float red[kWaves];
  __shared__ Teacher teach;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  const T* x = static_cast<const T*>(a.logits) + r * a.logits_stride;
  const Scale sc = scale_of(a.temperature);
  const int pieces = a.vocab / P, rest = a.vocab - pieces * P;
  load_teacher<THREADS>(a, r, teach);

  float m = -INFINITY, s[P] = {};
  for (int i = N * THREADS + tid; i < pieces; i += 2 * THREADS) {
    const bool two = i + THREADS < pieces;
    const u32x4 v0 = load_piece(x + (int64_t)i * P);
    const u32x4 v1 = two ? load_piece(x + (int64_t)(i + THREADS) * P) : u32x4(Elem<DT>::kMinusInf);
    float e0[P], e1[P];
    Elem<DT>::unpack(v0, e0);
    Elem<DT>::unpack(v1, e1);
    const float top = max_of(e1, max_of(e0, m)), base = top == -INFINITY ? 0.f : top;
    const float keep = sc.exp(m - base);
#pragma unroll
    for (int c = 0; c < P; ++c) s[c] = __builtin_fmaf(s[c], keep, sc.exp(e0[c] - base) + sc.exp(e1[c] - base));
    m = top;
  }
  u32x4 v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = u32x4(Elem<DT>::kMinusInf);
    if (i * THREADS + tid < pieces) v[i] = load_piece(x + (int64_t)(i * THREADS + tid) * P);
  }
  const float last = tid < rest ? Elem<DT>::load(x[(int64_t)pieces * P + tid]) : -INFINITY;
  float top = fmaxf(m, last);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i * THREADS < pieces) {
      float e[P];
      Elem<DT>::unpack(v[i], e);
      top = max_of(e, top);
    }
  top = block_max<kWaves>(top, red);
  const float keep = m == -INFINITY ? 0.f : sc.exp(m - top);
#pragma unroll
  for (int c = 0; c < P; ++c) s[c] *= keep;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i * THREADS < pieces) {
      float e[P];
      Elem<DT>::unpack(v[i], e);
#pragma unroll
      for (int c = 0; c < P; ++c) s[c] += sc.exp(e[c] - top);
    }
  const float z = block_sum<kWaves>(sum_of(s) + sc.exp(last - top), red);

  bool none;
  const float loss = teacher_loss<THREADS, DT>(a, sc, x, top, z, teach, red, &none);
  if (a.loss && tid == 0) a.loss[r] = loss;
  if (!a.grad) return;

  T* grad = static_cast<T*>(a.grad) + r * a.grad_stride;
  const float w = none ? 0.f : a.weight[r] * sc.inv, w_z = w / z;
  const bool zero = w == 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i * THREADS + tid < pieces) store_piece(grad + (int64_t)(i * THREADS + tid) * P, grad_piece<DT>(v[i], sc, top, w_z, zero));
  if (tid < rest) grad[(int64_t)pieces * P + tid] = Elem<DT>::store(zero ? 0.f : sc.exp(last - top) * w_z);
  for (int i = N * THREADS + tid; i < pieces; i += THREADS)
    store_piece(grad + (int64_t)i * P, grad_piece<DT>(load_piece(x + (int64_t)i * P), sc, top, w_z, zero));
  __syncthreads();
  if (!zero) teacher_grad<THREADS, DT>(a, sc, x, grad, top, z, w, teach, 0, a.vocab);
}

// Few rows: each is cut into parts of kPart pieces, one workgroup each. The first launch
// leaves every part's maximum and sum in the workspace, the second joins a row's parts,
// in order, and writes the gradient of its own part (and, part 0, the loss).
constexpr int kPartThreads = 256;
constexpr int kPartPieces = 4;  // a thread
constexpr int kPart = kPartThreads * kPartPieces;

struct PartStat {
  float top, sum;
};

template <int DT>
__device__ __forceinline__ void load_part(const DistillArgs& a, const typename Elem<DT>::type* x, int part,
                                          u32x4 (&v)[kPartPieces], float* last) {
  constexpr int P = Elem<DT>::kPiece;
  const int pieces = a.vocab / P;
#pragma unroll
  for (int i = 0; i < kPartPieces; ++i) {
    const int64_t p = (int64_t)part * kPart + i * kPartThreads + threadIdx.x;
    v[i] = u32x4(Elem<DT>::kMinusInf);
    if (p < pieces) v[i] = load_piece(x + p * P);
  }
  // The elements behind the last whole piece belong to part 0.
  const int64_t at = (int64_t)pieces * P + threadIdx.x;
  *last = part == 0 && at < a.vocab ? Elem<DT>::load(x[at]) : -INFINITY;
}

template <int DT>
__global__ __launch_bounds__(kPartThreads) void distill_part_kernel(DistillArgs a) {
  constexpr int P = Elem<DT>::kPiece, kWaves = kPartThreads / 64;
  __shared__ float red[kWaves];
  const int part = blockIdx.x;
  const int64_t r = blockIdx.y;
  const Scale sc = scale_of(a.temperature);
  u32x4 v[kPartPieces];
  float last;
  load_part<DT>(a, static_cast<const typename Elem<DT>::type*>(a.logits) + r * a.logits_stride, part, v, &last);
  float e[kPartPieces][P], top = last;
#pragma unroll
  for (int i = 0; i < kPartPieces; ++i) {
    Elem<DT>::unpack(v[i], e[i]);
    top = max_of(e[i], top);
  }
  top = block_max<kWaves>(top, red);
  const float base = top == -INFINITY ? 0.f : top;  // a part without weight adds nothing
  float s[P] = {};
#pragma unroll
  for (int i = 0; i < kPartPieces; ++i)
#pragma unroll
    for (int c = 0; c < P; ++c) s[c] += sc.exp(e[i][c] - base);
  const float z = block_sum<kWaves>(sum_of(s) + sc.exp(last - base), red);
  if (threadIdx.x == 0) static_cast<PartStat*>(a.workspace)[r * gridDim.x + part] = {top, z};
}

template <int DT>
__global__ __launch_bounds__(kPartThreads) void distill_join_kernel(DistillArgs a, int parts) {
  typedef typename Elem<DT>::type T;
  constexpr int P = Elem<DT>::kPiece, kWaves = kPartThreads / 64;
  __shared__ float red[kWaves];
  __shared__ Teacher teach;
  const int part = blockIdx.x, tid = threadIdx.x;
  const int64_t r = blockIdx.y;
  const T* x = static_cast<const T*>(a.logits) + r * a.logits_stride;
  const Scale sc = scale_of(a.temperature);
  u32x4 v[kPartPieces];
  float last;
  if (a.grad) load_part<DT>(a, x, part, v, &last);
  load_teacher<kPartThreads>(a, r, teach);
  const PartStat* stat = static_cast<const PartStat*>(a.workspace) + r * parts;
  float top = -INFINITY;
  for (int i = tid; i < parts; i += kPartThreads) top = fmaxf(top, stat[i].top);
  top = block_max<kWaves>(top, red);
  float z = 0.f;
  for (int i = tid; i < parts; i += kPartThreads) z += stat[i].sum * sc.exp(stat[i].top - top);
  z = block_sum<kWaves>(z, red);
  bool none;
  const float loss = teacher_loss<kPartThreads, DT>(a, sc, x, top, z, teach, red, &none);
  if (a.loss && tid == 0 && part == 0) a.loss[r] = loss;
  if (!a.grad) return;

  T* grad = static_cast<T*>(a.grad) + r * a.grad_stride;
  const float w = none ? 0.f : a.weight[r] * sc.inv, w_z = w / z;
  const bool zero = w == 0.f;
  const int pieces = a.vocab / P;
#pragma unroll
  for (int i = 0; i < kPartPieces; ++i) {
    const int64_t p = (int64_t)part * kPart + i * kPartThreads + tid;
    if (p < pieces) store_piece(grad + p * P, grad_piece<DT>(v[i], sc, top, w_z, zero));
  }
  const int64_t at = (int64_t)pieces * P + tid;
  if (part == 0 && at < a.vocab) grad[at] = Elem<DT>::store(zero ? 0.f : sc.exp(last - top) * w_z);
  __syncthreads();
  if (zero) return;
  const int64_t lo = (int64_t)part * kPart * P, hi = lo + (int64_t)kPart * P;
  teacher_grad<kPartThreads, DT>(a, sc, x, grad, top, z, w, teach, (int)lo, (int)(hi < pieces * (int64_t)P ? hi : pieces * (int64_t)P));
  if (part == 0) teacher_grad<kPartThreads, DT>(a, sc, x, grad, top, z, w, teach, pieces * P, a.vocab);
}

static int parts_of(int dtype, int vocab) {
  const int64_t pieces = vocab / (dtype == TF_DT_F32 ? 4 : 8);
  return (int)((pieces + kPart - 1) / kPart);
}

// Rows that one workgroup each leave too few workgroups for the chip are cut.
constexpr int kFewRows = 128;
constexpr int kMaxParts = 65535;
static bool cut(int dtype, int rows, int vocab) {
  return rows <= kFewRows && parts_of(dtype, vocab) > 2 && parts_of(dtype, vocab) <= kMaxParts;
}

template <int DT>
static void launch(const DistillArgs& a, hipStream_t stream) {
  const int parts = parts_of(DT, a.vocab);
  if (cut(DT, a.rows, a.vocab)) {
    hipLaunchKernelGGL(distill_part_kernel<DT>, dim3(parts, a.rows), dim3(kPartThreads), 0, stream, a);
    hipLaunchKernelGGL(distill_join_kernel<DT>, dim3(a.grad ? parts : 1, a.rows), dim3(kPartThreads), 0, stream, a, parts);
    return;
  }
  const int pieces = a.vocab / Elem<DT>::kPiece;
  const dim3 grid(a.rows);
  if (pieces <= 256 * 8)
    hipLaunchKernelGGL((distill_row_kernel<DT, 256, 8>), grid, dim3(256), 0, stream, a);
  else if (pieces <= 512 * 16)
    hipLaunchKernelGGL((distill_row_kernel<DT, 512, 16>), grid, dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((distill_row_kernel<DT, 1024, 16>), grid, dim3(1024), 0, stream, a);
}

size_t distill_workspace(int dtype, int rows, int vocab, int) {
  return cut(dtype, rows, vocab) ? ((size_t)rows * parts_of(dtype, vocab) * sizeof(PartStat) + 15) / 16 * 16 : 16;
}

hipError_t launch_distill(const DistillArgs& a, hipStream_t stream) {
  if (a.dtype == TF_DT_F32) launch<TF_DT_F32>(a, stream);
  if (a.dtype == TF_DT_F16) launch<TF_DT_F16>(a, stream);
  if (a.dtype == TF_DT_BF16) launch<TF_DT_BF16>(a, stream);
  return hipGetLastError();
}

}  // namespace tf_exl3
