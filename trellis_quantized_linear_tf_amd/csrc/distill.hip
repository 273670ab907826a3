// Distillation from a teacher's top logits: the loss of each row and its gradient.
#include <math.h>

#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxTop = 1024;

// One workgroup per row: maximum, sum of exponentials, the teacher's softmax, then the
// gradient, element by element, and at last the teacher's places again.
template <int DT>
__global__ __launch_bounds__(kThreads) void distill_kernel(DistillArgs a) {
  typedef typename Elem<DT>::type T;
  __shared__ float red[kWaves];
  __shared__ float tt[kMaxTop];
  __shared__ int at[kMaxTop];
  const int64_t r = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits) + r * a.logits_stride;
  const float inv = 1.f / a.temperature, c = kLog2e * inv;

  float ymax = -INFINITY;
  for (int j = threadIdx.x; j < a.top_k; j += kThreads) {
    const int i = a.index[r * a.top_k + j];
    const bool there = i >= 0 && i < a.vocab;
    at[j] = there ? i : -1;
    tt[j] = there ? load_elem(a.top, a.top_dtype, r * a.top_k + j) : -INFINITY;
    ymax = fmaxf(ymax, tt[j]);
  }
  ymax = block_max<kWaves>(ymax, red);
  float ysum = 0.f;
  for (int j = threadIdx.x; j < a.top_k; j += kThreads) ysum += at[j] >= 0 ? exp2f((tt[j] - ymax) * c) : 0.f;
  ysum = block_sum<kWaves>(ysum, red);
  const bool none = ysum == 0.f;

  float top = -INFINITY;
  for (int i = threadIdx.x; i < a.vocab; i += kThreads) top = fmaxf(top, Elem<DT>::load(x[i]));
  top = block_max<kWaves>(top, red);
  float z = 0.f;
  for (int i = threadIdx.x; i < a.vocab; i += kThreads) z += exp2f((Elem<DT>::load(x[i]) - top) * c);
  z = block_sum<kWaves>(z, red);
  const float lz = logf(z), lys = logf(ysum);

  float loss = 0.f;
  for (int j = threadIdx.x; j < a.top_k; j += kThreads) {
    float t = 0.f;
    if (at[j] >= 0) {
      const float ly = (tt[j] - ymax) * inv - lys;
      t = exp2f((tt[j] - ymax) * c) / ysum;
      if (t > 0.f) loss += t * (ly - ((Elem<DT>::load(x[at[j]]) - top) * inv - lz));
    }
    tt[j] = t;
  }
  loss = block_sum<kWaves>(loss, red);
  if (a.loss && threadIdx.x == 0) a.loss[r] = loss;
  if (!a.grad) return;

  T* grad = static_cast<T*>(a.grad) + r * a.grad_stride;
  const float w = none ? 0.f : a.weight[r] * inv;
  for (int i = threadIdx.x; i < a.vocab; i += kThreads)
    grad[i] = Elem<DT>::store(w == 0.f ? 0.f : exp2f((Elem<DT>::load(x[i]) - top) * c) / z * w);
  __syncthreads();
  if (w == 0.f) return;
  for (int j = threadIdx.x; j < a.top_k; j += kThreads) {
    if (at[j] < 0) continue;
    float t = 0.f;
    bool first = true;
    for (int i = 0; i < a.top_k; ++i)
      if (at[i] == at[j]) {
        first = first && i >= j;
        t += tt[i];
      }
    if (first) grad[at[j]] = Elem<DT>::store((exp2f((Elem<DT>::load(x[at[j]]) - top) * c) / z - t) * w);
  }
}

}  // namespace

size_t distill_workspace(int, int, int, int) { return 16; }

hipError_t launch_distill(const DistillArgs& a, hipStream_t stream) {
  const dim3 grid(a.rows), block(kThreads);
  if (a.dtype == TF_DT_F32) hipLaunchKernelGGL(distill_kernel<TF_DT_F32>, grid, block, 0, stream, a);
  if (a.dtype == TF_DT_F16) hipLaunchKernelGGL(distill_kernel<TF_DT_F16>, grid, block, 0, stream, a);
  if (a.dtype == TF_DT_BF16) hipLaunchKernelGGL(distill_kernel<TF_DT_BF16>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace tf_exl3
