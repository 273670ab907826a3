// Attention of a tree of drafted tokens over a paged cache.
#include <math.h>

#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

// One wave per (head, node, sequence). Lane l holds dimensions l, l + 64, ... of the
// query and of the running output; keys come one at a time, with the running maximum
// and sum of the softmax.
template <int DT>
__global__ __launch_bounds__(64) void tree_attention_kernel(tf_exl3_tree_attention_args a) {
  typedef typename Elem<DT>::type T;
  const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z, lane = threadIdx.x;
  const int g = h / (a.q_heads / a.kv_heads);
  const T* q = static_cast<const T*>(a.q) + b * a.q_stride[0] + i * a.q_stride[1] + h * a.q_stride[2];
  float qr[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 4; ++c) qr[c] = c * 64 + lane < a.head_dim ? Elem<DT>::load(q[c * 64 + lane]) : 0.f;
  const int64_t room = (int64_t)a.table_pages * a.page_size;
  int64_t len = a.lengths[b];
  len = len < 0 ? 0 : len > room ? room : len;
  const uint64_t seen = (uint64_t)a.mask[(int64_t)b * a.nodes + i];
  float m = -INFINITY, z = 0.f;
  for (int64_t j = 0; j < len + a.nodes; ++j) {
    const T *k, *v;
    if (j < len) {
      int page = a.table[b * a.table_stride + j / a.page_size];
      if (page < 0 || page >= a.pages) page = 0;
      const int64_t slot = j % a.page_size;
      k = static_cast<const T*>(a.k_cache) + page * a.k_cache_stride[0] + slot * a.k_cache_stride[1] +
          g * a.k_cache_stride[2];
      v = static_cast<const T*>(a.v_cache) + page * a.v_cache_stride[0] + slot * a.v_cache_stride[1] +
          g * a.v_cache_stride[2];
    } else {
      const int t = (int)(j - len);
      if (!((seen >> t) & 1)) continue;
      k = static_cast<const T*>(a.k) + b * a.k_stride[0] + t * a.k_stride[1] + g * a.k_stride[2];
      v = static_cast<const T*>(a.v) + b * a.v_stride[0] + t * a.v_stride[1] + g * a.v_stride[2];
    }
    float x = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c * 64 + lane < a.head_dim) x = __builtin_fmaf(qr[c], Elem<DT>::load(k[c * 64 + lane]), x);
    x = wave_sum(x) * a.scale;
    const float top = fmaxf(m, x);
    const float keep = m == -INFINITY ? 0.f : expf(m - top), p = expf(x - top);
    z = z * keep + p;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c * 64 + lane < a.head_dim) o[c] = __builtin_fmaf(p, Elem<DT>::load(v[c * 64 + lane]), o[c] * keep);
    m = top;
  }
  T* out = static_cast<T*>(a.out) + b * a.out_stride[0] + i * a.out_stride[1] + h * a.out_stride[2];
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c * 64 + lane < a.head_dim) out[c * 64 + lane] = Elem<DT>::store(z == 0.f ? 0.f : o[c] / z);
}

size_t tree_attention_workspace(const tf_exl3_tree_attention_args&) { return 16; }

hipError_t launch_tree_attention(const tf_exl3_tree_attention_args& a, hipStream_t stream) {
  const dim3 grid(a.q_heads, a.nodes, a.batch), block(64);
  if (a.dtype == TF_DT_F16)
    hipLaunchKernelGGL(tree_attention_kernel<TF_DT_F16>, grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL(tree_attention_kernel<TF_DT_BF16>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace tf_exl3
