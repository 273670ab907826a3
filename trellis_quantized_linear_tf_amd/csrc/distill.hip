// Distillation from a teacher's top logits: the loss of each row and its gradient.
//
// With d = x - max x, the student's p[i] = 2^(d c) / z, c = log2(e) / T, z their sum; a
// row's loss and gradient need z and the maximum before anything can be written, so a
// row is read, held on chip where it fits, and the gradient written from what is held.
// Bound by the logits' bytes, read once and, with the gradient, written once.
#include <math.h>

#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

constexpr int kMaxTop = 1024;
constexpr int kGroupElems = 16;  // held elements that are summed by one maximum

// 2^(d c) with c in two parts: the product's error is then one rounding of the
// exponent and not the rounding of c times |d|, which all elements would share.
struct Scale {
  float inv, c, c_low;
  __device__ float exp(float d) const { return __builtin_amdgcn_exp2f(__builtin_fmaf(d, c, d * c_low)); }
};

__device__ __forceinline__ Scale scale_of(const DistillArgs& a) { return {a.inv, a.c, a.c_low}; }

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

// A running maximum m and sums s of 2^((x - m) c), taken on by M pieces.
template <int DT, int M>
__device__ __forceinline__ void take(const u32x4* v, const Scale& sc, float& m, float (&s)[Elem<DT>::kPiece]) {
  constexpr int P = Elem<DT>::kPiece;
  float e[M][P], top = m;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    Elem<DT>::unpack(v[i], e[i]);
    top = max_of(e[i], top);
  }
  const float base = top == -INFINITY ? 0.f : top, keep = sc.exp(m - base);
#pragma unroll
  for (int c = 0; c < P; ++c) s[c] *= keep;
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int c = 0; c < P; ++c) s[c] += sc.exp(e[i][c] - base);
  m = top;
}

// The teacher's entries of a row. Its probabilities do not depend on the student: the first
// wave works them out while the row is on its way. In the gradient an entry is met again by
// the thread that writes the piece with its place, so each thread has a list of its entries.
template <int THREADS>
struct Teacher {
  float t[kMaxTop];  // probability
  int at[kMaxTop];   // place, -1 for an entry that is left out
  int next[kMaxTop], head[THREADS];
  int none;  // no entry at all
};

// The first wave's part. A lane's first entry is loaded ahead, into registers.
template <int DT>
struct Entries {
  typedef typename Elem<DT>::type T;
  int at0;
  float y0, x0;
  float ymax, ysum;

  __device__ __forceinline__ int place(const DistillArgs& a, int64_t r, int j) const {
    const int i = a.index[r * a.top_k + j];
    return i >= 0 && i < a.vocab ? i : -1;
  }
  __device__ __forceinline__ float logit(const DistillArgs& a, int64_t r, int j) const {
    return load_elem(a.top, a.top_dtype, r * a.top_k + j);
  }
  __device__ __forceinline__ void begin(const DistillArgs& a, int64_t r) {
    at0 = -1, y0 = x0 = 0.f;
    if ((int)threadIdx.x < a.top_k && threadIdx.x < 64) at0 = a.index[r * a.top_k + threadIdx.x], y0 = logit(a, r, threadIdx.x);
  }
  // Probabilities into shared memory; the student's logit at the first entry on its way.
  template <int THREADS>
  __device__ __forceinline__ void softmax(const DistillArgs& a, const Scale& sc, int64_t r, const T* x, Teacher<THREADS>& s) {
    const int lane = threadIdx.x;
    if (at0 >= a.vocab || at0 < 0) at0 = -1, y0 = -INFINITY;
    if (at0 >= 0) x0 = Elem<DT>::load(x[at0]);
    bool any = at0 >= 0;
    ymax = y0;
    if (lane < a.top_k) s.at[lane] = at0;
    for (int j = lane + 64; j < a.top_k; j += 64) {
      const int at = place(a, r, j);
      s.at[j] = at;
      s.t[j] = at >= 0 ? logit(a, r, j) : -INFINITY;
      any = any || at >= 0;
      ymax = fmaxf(ymax, s.t[j]);
    }
    ymax = wave_max(lane < a.top_k ? ymax : -INFINITY);
    const uint64_t some = __ballot(any);
    if (lane == 0) s.none = some == 0;
    ysum = at0 >= 0 ? sc.exp(y0 - ymax) : 0.f;
    for (int j = lane + 64; j < a.top_k; j += 64) ysum += s.at[j] >= 0 ? sc.exp(s.t[j] - ymax) : 0.f;
    ysum = wave_sum(ysum);
    if (lane < a.top_k) s.t[lane] = at0 >= 0 ? sc.exp(y0 - ymax) / ysum : 0.f;
    for (int j = lane + 64; j < a.top_k; j += 64) s.t[j] = s.at[j] >= 0 ? sc.exp(s.t[j] - ymax) / ysum : 0.f;
  }
  // The row's loss, in lane 63, given the student's maximum and sum.
  template <int THREADS>
  __device__ __forceinline__ float loss(const DistillArgs& a, const Scale& sc, int64_t r, const T* x, float top, float z,
                                        const Teacher<THREADS>& s) const {
    const int lane = threadIdx.x;
    const float lz = logf(z), lys = logf(ysum);
    auto term = [&](int j, float y, float xj) {
      const float t = s.t[j];
      return t > 0.f ? t * ((y - ymax) * sc.inv - lys - ((xj - top) * sc.inv - lz)) : t;  // a NaN stays one
    };
    float sum = at0 >= 0 ? term(lane, y0, x0) : 0.f;
    for (int j = lane + 64; j < a.top_k; j += 64)
      if (s.at[j] >= 0) sum += term(j, logit(a, r, j), Elem<DT>::load(x[s.at[j]]));
    return wave_scan(sum);
  }
};

// Entries with places in the pieces [lo, hi) into the lists of the threads that write them:
// the piece's number modulo THREADS, or a row's last elements in order. What is made of a
// list does not depend on its order. Entries without mass, as a padded list has them, change nothing and
// stay out.
template <int P, int THREADS>
__device__ __forceinline__ void link(const DistillArgs& a, Teacher<THREADS>& s, int pieces, int64_t lo, int64_t hi) {
  for (int j = threadIdx.x; j < a.top_k; j += THREADS) {
    const int at = s.at[j], piece = at / P;
    if (at < 0 || piece < lo || piece >= hi || s.t[j] == 0.f) continue;
    s.next[j] = atomicExch(&s.head[piece < pieces ? piece % THREADS : at - pieces * P], j);
  }
}

// What a thread writes of a row's gradient. Its pieces are numbered by `slot`.
template <int DT, int THREADS>
struct Writer {
  static constexpr int P = Elem<DT>::kPiece;
  const Scale sc;
  const Teacher<THREADS>& s;
  float top, z, w, w_z;
  bool zero;
  int first, at, next;  // the list's first entry
  float t;
  uint32_t slots;  // with an entry; 31 stands for all from 31 on

  __device__ __forceinline__ Writer(const Scale& scale, const Teacher<THREADS>& teach, float top_, float z_, float weight,
                                    int64_t lo)
      : sc(scale), s(teach), top(top_), z(z_), w(teach.none ? 0.f : weight * scale.inv), w_z(w / z_), zero(w == 0.f) {
    first = s.head[threadIdx.x], at = next = -1, t = 0.f, slots = 0;
    if (first >= 0) at = s.at[first], t = s.t[first], next = s.next[first];
    for (int j = first; j >= 0; j = s.next[j]) slots |= 1u << slot_of((int)((s.at[j] / P - lo) / THREADS));
  }
  __device__ static __forceinline__ int slot_of(int i) { return i < 31 ? i : 31; }

  // The teacher's mass at a place of the list: the sum of two does not depend on their order,
  // that of more is taken in units of 2^-62.
  __device__ __forceinline__ float mass(int place) const {
    float sum = 0.f;
    uint64_t units = 0;
    int n = 0;
    for (int j = first; j >= 0; j = s.next[j])
      if (s.at[j] == place) {
        sum += s.t[j];
        units += (uint64_t)((double)s.t[j] * 0x1p62);
        ++n;
      }
    return n > 2 && sum == sum ? (float)((double)units * 0x1p-62) : sum;
  }
  __device__ __forceinline__ float at_place(float x, float mass) const { return (sc.exp(x - top) / z - mass) * w; }
  __device__ __forceinline__ void fix(const float (&x)[P], float (&g)[P], int c, float mass) const {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i == c) g[i] = at_place(x[i], mass);
  }
  __device__ __forceinline__ u32x4 operator()(u32x4 v, int64_t p, int slot) const {
    if (zero) return u32x4(0u);  // whatever the row holds
    float x[P], g[P];
    Elem<DT>::unpack(v, x);
#pragma unroll
    for (int c = 0; c < P; ++c) g[c] = sc.exp(x[c] - top) * w_z;
    if ((slots >> slot_of(slot)) & 1) {
      if (next < 0) {
        if (at / P == p) fix(x, g, at % P, t);
      } else {
        // Each place once, so that a list of n entries of one place takes n steps a walk and not n^2 (1024
        // entries at one place of 129280, 16 rows: 138 ms before).
        uint32_t done = 0;
        for (int j = first; j >= 0; j = s.next[j]) {
          const int place = s.at[j], c = place % P;
          if (place / P != p || (done >> c) & 1) continue;
          done |= 1u << c;
          fix(x, g, c, mass(place));
        }
      }
    }
    return Elem<DT>::pack(g);
  }
  // The thread's element behind the whole pieces, at `place`.
  __device__ __forceinline__ typename Elem<DT>::type last(float x, int64_t place) const {
    if (zero) return Elem<DT>::store(0.f);
    return Elem<DT>::store(at_place(x, mass((int)place)));
  }
};

// One workgroup per row, N pieces of 16 bytes held by each thread; what a longer row has
// beyond them is read first, with a running maximum, and once more for the gradient
// (then from the memory-side cache: the rows in flight are below its 256 MB). The
// sums' order depends on the row's length alone, so the loss has the same bits with and
// without the gradient. 4096 rows of 129280 bf16, loss and gradient: 2.12 GB in 416 us, 5.1
// TB/s, the rate of a copy; reading the row twice instead measured 1.9 ms with one element a
// thread, summing it only after the last piece had come 536 us.
template <int DT, int THREADS, int N>
__global__ __launch_bounds__(THREADS, 4) void distill_row_kernel(DistillArgs a) {
  typedef typename Elem<DT>::type T;
  constexpr int P = Elem<DT>::kPiece, kWaves = THREADS / 64;
  __shared__ float red[kWaves];
  __shared__ Teacher<THREADS> teach;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  const T* x = static_cast<const T*>(a.logits) + r * a.logits_stride;
  const Scale sc = scale_of(a);
  const int pieces = a.vocab / P, rest = a.vocab - pieces * P;
  Entries<DT> entries;
  entries.begin(a, r);
  teach.head[tid] = -1;

  float m = -INFINITY, s[P] = {};
  for (int i = N * THREADS + tid; i < pieces; i += 2 * THREADS) {
    u32x4 v[2];
    v[0] = load_piece(x + (int64_t)i * P);
    v[1] = i + THREADS < pieces ? load_piece(x + (int64_t)(i + THREADS) * P) : u32x4(Elem<DT>::kMinusInf);
    take<DT, 2>(v, sc, m, s);
  }
  u32x4 v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = u32x4(Elem<DT>::kMinusInf);
    if (i * THREADS + tid < pieces) v[i] = load_piece(x + (int64_t)(i * THREADS + tid) * P);
  }
  const float last = tid < rest ? Elem<DT>::load(x[(int64_t)pieces * P + tid]) : -INFINITY;
  if (tid < 64) entries.softmax(a, sc, r, x, teach);
  // Pieces are summed as they come, by the thread's own maximum so far, so that this is
  // done while the later ones are on their way.
  constexpr int kGroup = kGroupElems / P;
#pragma unroll
  for (int g = 0; g < N; g += kGroup)
    if (g * THREADS < pieces) take<DT, kGroup>(v + g, sc, m, s);
  const float top = block_max<kWaves>(fmaxf(m, last), red);
  if (a.grad) link<P, THREADS>(a, teach, pieces, 0, (int64_t)pieces + 1);
  const float keep = m == -INFINITY ? 0.f : sc.exp(m - top);
#pragma unroll
  for (int c = 0; c < P; ++c) s[c] *= keep;
  const float z = block_sum<kWaves>(sum_of(s) + sc.exp(last - top), red);

  if (tid < 64 && a.loss) {
    const float loss = entries.loss(a, sc, r, x, top, z, teach);
    if (tid == 63) a.loss[r] = loss;
  }
  if (!a.grad) return;

  T* grad = static_cast<T*>(a.grad) + r * a.grad_stride;
  const Writer<DT, THREADS> out(sc, teach, top, z, a.weight[r], 0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int p = i * THREADS + tid;
    if (p < pieces) store_piece(grad + (int64_t)p * P, out(v[i], p, i));
  }
  if (tid < rest) grad[(int64_t)pieces * P + tid] = out.last(last, (int64_t)pieces * P + tid);
  for (int i = N * THREADS + tid; i < pieces; i += THREADS)
    store_piece(grad + (int64_t)i * P, out(load_piece(x + (int64_t)i * P), i, i / THREADS));
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
  const Scale sc = scale_of(a);
  u32x4 v[kPartPieces];
  float last;
  load_part<DT>(a, static_cast<const typename Elem<DT>::type*>(a.logits) + r * a.logits_stride, part, v, &last);
  float m = -INFINITY, s[P] = {};
  take<DT, kPartPieces>(v, sc, m, s);
  const float top = block_max<kWaves>(fmaxf(m, last), red);
  const float base = top == -INFINITY ? 0.f : top;  // a part without weight adds nothing
  const float keep = m == -INFINITY ? 0.f : sc.exp(m - base);
  const float z = block_sum<kWaves>(sum_of(s) * keep + sc.exp(last - base), red);
  if (threadIdx.x == 0) static_cast<PartStat*>(a.workspace)[r * gridDim.x + part] = {top, z};
}

template <int DT>
__global__ __launch_bounds__(kPartThreads) void distill_join_kernel(DistillArgs a, int parts) {
  typedef typename Elem<DT>::type T;
  constexpr int P = Elem<DT>::kPiece, kWaves = kPartThreads / 64;
  __shared__ float red[kWaves];
  __shared__ Teacher<kPartThreads> teach;
  const int part = blockIdx.x, tid = threadIdx.x;
  const int64_t r = blockIdx.y;
  const T* x = static_cast<const T*>(a.logits) + r * a.logits_stride;
  const Scale sc = scale_of(a);
  const int pieces = a.vocab / P;
  Entries<DT> entries;
  entries.begin(a, r);
  teach.head[tid] = -1;
  const PartStat* stat = static_cast<const PartStat*>(a.workspace) + r * parts;
  PartStat mine = {-INFINITY, 0.f};
  if (tid < parts) mine = stat[tid];
  u32x4 v[kPartPieces];
  float last = -INFINITY;
  if (a.grad) load_part<DT>(a, x, part, v, &last);
  if (tid < 64) entries.softmax(a, sc, r, x, teach);
  float top = mine.top;
  for (int i = tid + kPartThreads; i < parts; i += kPartThreads) top = fmaxf(top, stat[i].top);
  top = block_max<kWaves>(top, red);
  const int64_t lo = (int64_t)part * kPart, hi = lo + kPart < pieces ? lo + kPart : pieces;
  if (a.grad) {
    link<P, kPartThreads>(a, teach, pieces, lo, hi);
    if (part == 0) link<P, kPartThreads>(a, teach, pieces, pieces, (int64_t)pieces + 1);
  }
  float z = tid < parts ? mine.sum * sc.exp(mine.top - top) : 0.f;
  for (int i = tid + kPartThreads; i < parts; i += kPartThreads) z += stat[i].sum * sc.exp(stat[i].top - top);
  z = block_sum<kWaves>(z, red);
  if (tid < 64 && part == 0 && a.loss) {
    const float loss = entries.loss(a, sc, r, x, top, z, teach);
    if (tid == 63) a.loss[r] = loss;
  }
  if (!a.grad) return;

  T* grad = static_cast<T*>(a.grad) + r * a.grad_stride;
  const Writer<DT, kPartThreads> out(sc, teach, top, z, a.weight[r], lo);
#pragma unroll
  for (int i = 0; i < kPartPieces; ++i) {
    const int64_t p = lo + i * kPartThreads + tid;
    if (p < pieces) store_piece(grad + p * P, out(v[i], p, i));
  }
  const int64_t at = (int64_t)pieces * P + tid;
  if (part == 0 && at < a.vocab) grad[at] = out.last(last, at);
}

static int parts_of(int dtype, int vocab) {
  const int64_t pieces = vocab / (dtype == TF_DT_F32 ? 4 : 8);
  return (int)((pieces + kPart - 1) / kPart);
}

// Rows are cut where they are long (a workgroup of 1024, alone on its CU, would take one) and
// either together no more than the second launch finds in the caches, or so few that most
// CUs would have none. Rows of 129280, loss and
// gradient, cut against whole, us: fp32 16 rows 14.9 / 22.8, 64 17.6 / 26.4, 100 27.6 / 26.9,
// 256 63 / 52; bf16 16 rows 15.3 / 20.3, 128 21.2 / 25.0, 160 26.8 / 26.0, 256 38 / 30. Rows of
// 20000 whole 13 / 15 at any number.
constexpr int kLongRow = 512 * 16;         // pieces
constexpr int64_t kFewBytes = 40ll << 20;  // of logits
constexpr int kFewRows = 64;
static bool cut(int dtype, int rows, int vocab) {
  const int64_t bytes = (int64_t)vocab * (dtype == TF_DT_F32 ? 4 : 2);
  return bytes / 16 > kLongRow && (rows <= kFewRows || rows * bytes <= kFewBytes);
}

// Threads that hold a row between them.
static int row_threads(int dtype, int vocab) {
  const int pieces = vocab / (dtype == TF_DT_F32 ? 4 : 8);
  return pieces <= 256 * 8 ? 256 : pieces <= kLongRow ? 512 : 1024;
}

bool distill_fits(int dtype, int rows, int vocab) {
  return cut(dtype, rows, vocab) || launchable(rows, row_threads(dtype, vocab));
}

template <int DT>
static void launch(const DistillArgs& a, hipStream_t stream) {
  const int parts = parts_of(DT, a.vocab);
  if (cut(DT, a.rows, a.vocab)) {
    hipLaunchKernelGGL(distill_part_kernel<DT>, dim3(parts, a.rows), dim3(kPartThreads), 0, stream, a);
    hipLaunchKernelGGL(distill_join_kernel<DT>, dim3(a.grad ? parts : 1, a.rows), dim3(kPartThreads), 0, stream, a, parts);
    return;
  }
  const int threads = row_threads(DT, a.vocab);
  const dim3 grid(a.rows);
  if (threads == 256)
    hipLaunchKernelGGL((distill_row_kernel<DT, 256, 8>), grid, dim3(256), 0, stream, a);
  else if (threads == 512)
    hipLaunchKernelGGL((distill_row_kernel<DT, 512, 16>), grid, dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((distill_row_kernel<DT, 1024, 16>), grid, dim3(1024), 0, stream, a);
}

size_t distill_workspace(int dtype, int rows, int vocab, int) {
  return cut(dtype, rows, vocab) ? ((size_t)rows * parts_of(dtype, vocab) * sizeof(PartStat) + 15) / 16 * 16 : 16;
}

hipError_t launch_distill(const DistillArgs& args, hipStream_t stream) {
  DistillArgs a = args;
  const double c = 1.4426950408889634 / (double)a.temperature;
  a.inv = 1.f / a.temperature, a.c = (float)c;
  // The low part is above 0, so that a difference of -inf meets no +inf and no 0 in it.
  if ((double)a.c > c) a.c = nextafterf(a.c, 0.f);
  a.c_low = fmaxf((float)(c - (double)a.c), 1.2e-38f);
  if (a.dtype == TF_DT_F32) launch<TF_DT_F32>(a, stream);
  if (a.dtype == TF_DT_F16) launch<TF_DT_F16>(a, stream);
  if (a.dtype == TF_DT_BF16) launch<TF_DT_BF16>(a, stream);
  return hipGetLastError();
}

}  // namespace tf_exl3
