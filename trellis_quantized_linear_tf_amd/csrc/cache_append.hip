// Rows of keys and values into a paged cache, byte for byte.
#include "ops_device.hpp"
#include "ops_launch.hpp"

namespace tf_exl3 {

// One workgroup per (token, sequence): every head's row of k and v.
template <typename T>
__global__ __launch_bounds__(256) void cache_append_kernel(tf_exl3_cache_append_args a) {
  const int j = blockIdx.x, b = blockIdx.y;
  int count = a.counts ? a.counts[b] : a.tokens;
  if (j >= count) return;
  const int t = a.nodes ? a.nodes[(int64_t)b * a.tokens + j] : j;
  const int64_t pos = (int64_t)a.lengths[b] + j;
  if (t < 0 || t >= a.tokens || pos < 0 || pos >= (int64_t)a.table_pages * a.page_size) return;
  const int page = a.table[b * a.table_stride + pos / a.page_size];
  if (page < 0 || page >= a.pages) return;
  const int64_t slot = pos % a.page_size;
  const T* k = static_cast<const T*>(a.k) + b * a.k_stride[0] + t * a.k_stride[1];
  const T* v = static_cast<const T*>(a.v) + b * a.v_stride[0] + t * a.v_stride[1];
  T* kc = static_cast<T*>(a.k_cache) + page * a.k_cache_stride[0] + slot * a.k_cache_stride[1];
  T* vc = static_cast<T*>(a.v_cache) + page * a.v_cache_stride[0] + slot * a.v_cache_stride[1];
  for (int i = threadIdx.x; i < a.kv_heads * a.head_dim; i += 256) {
    const int h = i / a.head_dim, d = i % a.head_dim;
    kc[h * a.k_cache_stride[2] + d] = k[h * a.k_stride[2] + d];
    vc[h * a.v_cache_stride[2] + d] = v[h * a.v_stride[2] + d];
  }
}

hipError_t launch_cache_append(const tf_exl3_cache_append_args& a, hipStream_t stream) {
  const dim3 grid(a.tokens, a.batch), block(256);
  if (a.elem_bytes == 1) hipLaunchKernelGGL(cache_append_kernel<uint8_t>, grid, block, 0, stream, a);
  if (a.elem_bytes == 2) hipLaunchKernelGGL(cache_append_kernel<uint16_t>, grid, block, 0, stream, a);
  if (a.elem_bytes == 4) hipLaunchKernelGGL(cache_append_kernel<uint32_t>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace tf_exl3
