// Verification of drafted tokens against the target's logits, from given random numbers.
#include <math.h>

#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// Rank of a logit: -inf and NaN have none.
template <int DT>
__device__ __forceinline__ float logit(const void* row, int i) {
  const float x = Elem<DT>::load(static_cast<const typename Elem<DT>::type*>(row)[i]);
  return x == x ? x : -INFINITY;
}

// Weight of logit x in a row of maximum top at temperature t > 0. The difference to an
// infinite maximum is taken as 0 for the places that reach it.
__device__ __forceinline__ double weight_of(float x, float top, double t) {
  if (x == top) return 1.0;
  if (x == -INFINITY || top == INFINITY) return 0.0;
  return exp(((double)x - (double)top) / t);
}

// First place, over a workgroup, whose running sum of f(i) is over u times the sum.
template <typename F>
__device__ int sample_row(F f, int vocab, double u, double* sums, int* found) {
  // Thread-contiguous pieces: the sum of each, then the piece that crosses, in order.
  const int piece = (vocab + kThreads - 1) / kThreads;
  const int lo = min(vocab, (int)threadIdx.x * piece), hi = min(vocab, lo + piece);
  double s = 0.0;
  for (int i = lo; i < hi; ++i) s += f(i);
  __syncthreads();
  sums[threadIdx.x] = s;
  if (threadIdx.x == 0) *found = -1;
  __syncthreads();
  double before = 0.0, total = 0.0;
  int last = -1, mine = -1;
  for (int j = 0; j < kThreads; ++j) {
    if (j == (int)threadIdx.x) before = total;
    total += sums[j];
    if (sums[j] > 0.0) last = j;
  }
  const double goal = u * total;
  if (s > 0.0 && (before + s > goal || (int)threadIdx.x == last) && !(before > goal)) {
    double c = before;
    for (int i = lo; i < hi; ++i) {
      const double w = f(i);
      c += w;
      if (w > 0.0) mine = i;
      if (c > goal) break;
    }
  }
  // The first piece that crosses holds the place.
  if (mine >= 0) atomicMin(reinterpret_cast<unsigned*>(found), (unsigned)mine);
  __syncthreads();
  return *found;
}

__device__ __forceinline__ double fraction(float u) { return u > 0.f ? (double)u : 0.0; }

// One workgroup per row: its token.
template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(VerifyArgs a, int32_t* token) {
  __shared__ float smax[kWaves];
  __shared__ double sums[kThreads];
  __shared__ int found;
  const int i = blockIdx.x, b = blockIdx.y;
  const auto* row = static_cast<const typename Elem<DT>::type*>(a.logits) + b * a.stride_batch + i * a.stride_node;
  float top = -INFINITY;
  for (int j = threadIdx.x; j < a.vocab; j += kThreads) top = fmaxf(top, logit<DT>(row, j));
  top = block_max<kWaves>(top, smax);
  const float t = a.temperature ? a.temperature[b] : 1.f;
  int place = -1;
  if (top != -INFINITY) {
    if (t > 0.f) {
      place = sample_row([&](int j) { return weight_of(logit<DT>(row, j), top, t); }, a.vocab,
                         fraction(a.u[(int64_t)b * a.nodes + i]), sums, &found);
    } else {
      place = sample_row([&](int j) { return logit<DT>(row, j) == top ? 1.0 : 0.0; }, a.vocab, 0.0, sums, &found);
    }
  }
  if (threadIdx.x == 0) token[(int64_t)b * a.nodes + i] = place;
}

// One thread per sequence walks its tree.
__global__ __launch_bounds__(64) void walk_kernel(VerifyArgs a, const int32_t* token) {
  const int b = blockIdx.x * 64 + threadIdx.x;
  if (b >= a.batch) return;
  const int64_t at = (int64_t)b * a.nodes;
  int node = 0, count = 0;
  for (int c = 1; c <= a.nodes; ++c) {
    if (c < a.nodes && !(a.parents[at + c] == node && a.tokens[at + c] == token[at + node] && token[at + node] >= 0)) continue;
    a.accepted[at + count++] = node;
    if (c < a.nodes) node = c;
  }
  a.count[b] = count;
  a.next[b] = token[at + node];
  for (int c = count; c < a.nodes; ++c) a.accepted[at + c] = -1;
}

// One workgroup per sequence: the chain's rows in turn.
template <int DT>
__global__ __launch_bounds__(kThreads) void chain_kernel(VerifyArgs a) {
  __shared__ float smax[kWaves];
  __shared__ double ssum[kWaves];
  __shared__ double sums[kThreads];
  __shared__ int found;
  const int b = blockIdx.x;
  const float t = a.temperature ? a.temperature[b] : 1.f;
  const int64_t at = (int64_t)b * a.nodes;
  for (int j = 0; j < a.nodes; ++j) {
    const auto* row = static_cast<const typename Elem<DT>::type*>(a.logits) + b * a.stride_batch + j * a.stride_node;
    float top = -INFINITY;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) top = fmaxf(top, logit<DT>(row, i));
    top = block_max<kWaves>(top, smax);
    int first = 0x7FFFFFFF;  // the first place of the maximum
    for (int i = threadIdx.x; i < a.vocab; i += kThreads)
      if (logit<DT>(row, i) == top) first = min(first, i);
    __syncthreads();
    if (threadIdx.x == 0) found = 0x7FFFFFFF;
    __syncthreads();
    atomicMin(&found, first);
    __syncthreads();
    first = found;
    auto w = [&](int i) {
      if (top == -INFINITY) return 0.0;
      if (!(t > 0.f)) return i == first ? 1.0 : 0.0;
      return weight_of(logit<DT>(row, i), top, t);
    };
    double z = 0.0;
    for (int i = threadIdx.x; i < a.vocab; i += kThreads) z += w(i);
    z = block_sum<kWaves>(z, ssum);
    const float* q = a.q + b * a.q_stride_batch + j * a.q_stride_node;
    if (j + 1 < a.nodes) {
      const int x = a.tokens[at + j + 1];
      const bool ok = x >= 0 && x < a.vocab && z > 0.0 &&
                      fraction(a.u[at + j]) * (double)q[x] < w(x) / z;
      if (ok) continue;
    }
    const bool rest = j + 1 < a.nodes;
    auto residual = [&](int i) {
      const double p = z > 0.0 ? w(i) / z : 0.0;
      const double r = p - (rest ? (double)q[i] : 0.0);
      return r > 0.0 ? r : 0.0;
    };
    const double u = fraction(a.u[at + a.nodes - 1]);
    int place = sample_row(residual, a.vocab, u, sums, &found);
    if (place < 0 && rest) {
      __syncthreads();
      place = sample_row([&](int i) { return z > 0.0 ? w(i) / z : 0.0; }, a.vocab, u, sums, &found);
    }
    if (threadIdx.x == 0) {
      a.count[b] = j + 1;
      a.next[b] = place;
    }
    return;
  }
}

template <int DT>
void launch(const VerifyArgs& a, hipStream_t stream) {
  if (a.q == nullptr && a.parents != nullptr) {
    int32_t* token = static_cast<int32_t*>(a.workspace);
    hipLaunchKernelGGL(sample_kernel<DT>, dim3(a.nodes, a.batch), dim3(kThreads), 0, stream, a, token);
    hipLaunchKernelGGL(walk_kernel, dim3((a.batch + 63) / 64), dim3(64), 0, stream, a, token);
  } else {
    hipLaunchKernelGGL(chain_kernel<DT>, dim3(a.batch), dim3(kThreads), 0, stream, a);
  }
}

}  // namespace

size_t verify_workspace(int batch, int nodes, int) { return ((size_t)batch * nodes * 4 + 15) / 16 * 16; }

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream) {
  if (a.dtype == TF_DT_F32) launch<TF_DT_F32>(a, stream);
  if (a.dtype == TF_DT_F16) launch<TF_DT_F16>(a, stream);
  if (a.dtype == TF_DT_BF16) launch<TF_DT_BF16>(a, stream);
  return hipGetLastError();
}

}  // namespace tf_exl3
