// C ABI of the operators around the projection: argument checks on the host, then one
// call into the launch interface. Nothing is launched or written on a refusal.
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "ops_launch.hpp"
#include "tf_exl3.h"

namespace {

constexpr int kMaxBatch = 65535;        // sequences, a grid dimension
constexpr int kMaxTreeNodes = 64;       // bits of a node's mask
constexpr int kMaxVerifyNodes = 1024;
constexpr int kMaxTop = 1024;           // the teacher's entries, held in shared memory
constexpr int64_t kMaxStride = 1ll << 40;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

size_t elem_size(int dt) { return dt == TF_DT_F32 ? 4 : 2; }

bool dtype_ok(int dt) { return dt == TF_DT_F32 || dt == TF_DT_F16 || dt == TF_DT_BF16; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (na == 0 || nb == 0 || a == nullptr || b == nullptr) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

// Bytes from the first to past the last element of [n0][n1][n2][d] with strides s.
size_t extent(int64_t n0, int64_t n1, int64_t n2, int64_t d, const int64_t* s, size_t elem) {
  return (size_t)((n0 - 1) * s[0] + (n1 - 1) * s[1] + (n2 - 1) * s[2] + d) * elem;
}

// A stride over a dimension of 1 is never used, whatever it is.
void settle(int64_t n0, int64_t n1, int64_t n2, int64_t* s) {
  if (n0 <= 1) s[0] = 0;
  if (n1 <= 1) s[1] = 0;
  if (n2 <= 1) s[2] = 0;
}

bool strides_ok(const int64_t* s, int64_t multiple) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] > kMaxStride || s[i] % multiple != 0) return false;
  return true;
}

// Rows that are written may not share elements: no stride of 0 over more than one of them.
bool apart(int64_t n0, int64_t n1, int64_t n2, const int64_t* s) {
  return (n0 <= 1 || s[0] != 0) && (n1 <= 1 || s[1] != 0) && (n2 <= 1 || s[2] != 0);
}

int cache_sizes(int pages, int page_size, int table_pages, int64_t table_stride) {
  if (pages < 1 || page_size < 1 || table_pages < 0 || table_stride < 0 || table_stride > kMaxStride) return TF_E_SIZE;
  // Positions are 32-bit: room for the longest sequence and its new tokens.
  if ((int64_t)table_pages * page_size > (1ll << 30)) return TF_E_SIZE;
  return TF_OK;
}

int attention_sizes(const tf_exl3_tree_attention_args* a) {
  if (a->dtype != TF_DT_F16 && a->dtype != TF_DT_BF16) return TF_E_DTYPE;
  if (a->batch < 0 || a->batch > kMaxBatch || a->nodes < 1 || a->nodes > kMaxTreeNodes) return TF_E_SIZE;
  if (a->kv_heads < 1 || a->q_heads < 1 || a->q_heads > kMaxBatch || a->q_heads % a->kv_heads != 0) return TF_E_SIZE;
  if (a->head_dim < 16 || a->head_dim > 256 || a->head_dim % 16 != 0) return TF_E_SIZE;
  const int st = cache_sizes(1, a->page_size, a->table_pages, 0);
  return st != TF_OK || tf_exl3::tree_attention_fits(*a) ? st : TF_E_SIZE;
}

int verify_sizes(int batch, int nodes, int vocab, bool tree) {
  if (batch < 0 || batch > kMaxBatch || nodes < 1 || nodes > kMaxVerifyNodes || vocab < 1) return TF_E_SIZE;
  return tf_exl3::verify_fits(batch, nodes, vocab, tree) ? TF_OK : TF_E_SIZE;
}

bool row_strides_ok(int64_t batch, int64_t node) {
  return batch >= 0 && node >= 0 && batch <= kMaxStride && node <= kMaxStride;
}

}  // namespace

extern "C" {

size_t tf_exl3_tree_attention_workspace(const tf_exl3_tree_attention_args* a) {
  if (a == nullptr || attention_sizes(a) != TF_OK) return 0;
  return tf_exl3::tree_attention_workspace(*a);
}

int tf_exl3_tree_attention(const tf_exl3_tree_attention_args* args, void* stream) {
  if (args == nullptr) return TF_E_NULL;
  tf_exl3_tree_attention_args settled = *args;
  tf_exl3_tree_attention_args* a = &settled;
  settle(a->batch, a->nodes, a->q_heads, a->q_stride);
  settle(a->batch, a->nodes, a->kv_heads, a->k_stride);
  settle(a->batch, a->nodes, a->kv_heads, a->v_stride);
  settle(a->pages, a->page_size, a->kv_heads, a->k_cache_stride);
  settle(a->pages, a->page_size, a->kv_heads, a->v_cache_stride);
  settle(a->batch, a->nodes, a->q_heads, a->out_stride);
  int st = attention_sizes(a);
  if (st == TF_OK) st = cache_sizes(a->pages, a->page_size, a->table_pages, a->table_stride);
  if (st != TF_OK) return st;
  if (!isfinite(a->scale)) return TF_E_SIZE;
  if (!strides_ok(a->q_stride, 8) || !strides_ok(a->k_stride, 8) || !strides_ok(a->v_stride, 8) ||
      !strides_ok(a->k_cache_stride, 8) || !strides_ok(a->v_cache_stride, 8) || !strides_ok(a->out_stride, 4) ||
      !apart(a->batch, a->nodes, a->q_heads, a->out_stride))
    return TF_E_SIZE;
  if (a->batch == 0) return TF_OK;
  if (!a->q || !a->k || !a->v || !a->mask || !a->k_cache || !a->v_cache || !a->lengths || !a->out || !a->workspace ||
      (a->table_pages > 0 && !a->table))
    return TF_E_NULL;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->k_cache, 16) ||
      !aligned(a->v_cache, 16) || !aligned(a->out, 8) || !aligned(a->workspace, 16) || !aligned(a->mask, 8) ||
      !aligned(a->table, 4) || !aligned(a->lengths, 4))
    return TF_E_ALIGN;
  const size_t need = tf_exl3::tree_attention_workspace(*a);
  if (a->workspace_bytes < need) return TF_E_WORKSPACE;
  const size_t rows_q = extent(a->batch, a->nodes, a->q_heads, a->head_dim, a->q_stride, 2);
  const size_t rows_k = extent(a->batch, a->nodes, a->kv_heads, a->head_dim, a->k_stride, 2);
  const size_t rows_v = extent(a->batch, a->nodes, a->kv_heads, a->head_dim, a->v_stride, 2);
  const size_t kc = extent(a->pages, a->page_size, a->kv_heads, a->head_dim, a->k_cache_stride, 2);
  const size_t vc = extent(a->pages, a->page_size, a->kv_heads, a->head_dim, a->v_cache_stride, 2);
  const size_t no = extent(a->batch, a->nodes, a->q_heads, a->head_dim, a->out_stride, 2);
  const void* written[2] = {a->out, a->workspace};
  const size_t bytes[2] = {no, need};
  for (int i = 0; i < 2; ++i) {
    const void* w = written[i];
    const size_t n = bytes[i];
    if (overlap(w, n, a->q, rows_q) || overlap(w, n, a->k, rows_k) || overlap(w, n, a->v, rows_v) ||
        overlap(w, n, a->k_cache, kc) || overlap(w, n, a->v_cache, vc) ||
        overlap(w, n, a->mask, (size_t)a->batch * a->nodes * 8) || overlap(w, n, a->lengths, (size_t)a->batch * 4) ||
        overlap(w, n, a->table, (size_t)((a->batch - 1) * a->table_stride + a->table_pages) * 4))
      return TF_E_ALIAS;
  }
  if (overlap(a->out, no, a->workspace, need)) return TF_E_ALIAS;
  const hipError_t e = tf_exl3::launch_tree_attention(*a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TF_OK : TF_E_LAUNCH;
}

int tf_exl3_cache_append(const tf_exl3_cache_append_args* args, void* stream) {
  if (args == nullptr) return TF_E_NULL;
  tf_exl3_cache_append_args settled = *args;
  tf_exl3_cache_append_args* a = &settled;
  settle(a->batch, a->tokens, a->kv_heads, a->k_stride);
  settle(a->batch, a->tokens, a->kv_heads, a->v_stride);
  settle(a->pages, a->page_size, a->kv_heads, a->k_cache_stride);
  settle(a->pages, a->page_size, a->kv_heads, a->v_cache_stride);
  if (a->elem_bytes != 1 && a->elem_bytes != 2 && a->elem_bytes != 4) return TF_E_DTYPE;
  if (a->batch < 0 || a->batch > kMaxBatch || a->tokens < 0 || a->tokens > (1 << 30) || a->kv_heads < 1 ||
      a->head_dim < 1 || (int64_t)a->kv_heads * a->head_dim > (1 << 24))
    return TF_E_SIZE;
  const int st = cache_sizes(a->pages, a->page_size, a->table_pages, a->table_stride);
  if (st != TF_OK) return st;
  if (!strides_ok(a->k_stride, 1) || !strides_ok(a->v_stride, 1) || !strides_ok(a->k_cache_stride, 1) ||
      !strides_ok(a->v_cache_stride, 1) || !apart(a->pages, a->page_size, a->kv_heads, a->k_cache_stride) ||
      !apart(a->pages, a->page_size, a->kv_heads, a->v_cache_stride))
    return TF_E_SIZE;
  if (!tf_exl3::cache_append_fits(*a)) return TF_E_SIZE;
  if (a->batch == 0 || a->tokens == 0 || a->table_pages == 0) return TF_OK;
  if (!a->k || !a->v || !a->k_cache || !a->v_cache || !a->table || !a->lengths) return TF_E_NULL;
  const uintptr_t e = (uintptr_t)a->elem_bytes;
  if (!aligned(a->k, e) || !aligned(a->v, e) || !aligned(a->k_cache, e) || !aligned(a->v_cache, e) ||
      !aligned(a->table, 4) || !aligned(a->lengths, 4) || !aligned(a->nodes, 4) || !aligned(a->counts, 4))
    return TF_E_ALIGN;
  const size_t nk = extent(a->batch, a->tokens, a->kv_heads, a->head_dim, a->k_stride, e);
  const size_t nv = extent(a->batch, a->tokens, a->kv_heads, a->head_dim, a->v_stride, e);
  const void* caches[2] = {a->k_cache, a->v_cache};
  const size_t bytes[2] = {extent(a->pages, a->page_size, a->kv_heads, a->head_dim, a->k_cache_stride, e),
                           extent(a->pages, a->page_size, a->kv_heads, a->head_dim, a->v_cache_stride, e)};
  for (int i = 0; i < 2; ++i) {
    if (overlap(caches[i], bytes[i], a->k, nk) || overlap(caches[i], bytes[i], a->v, nv) ||
        overlap(caches[i], bytes[i], a->table, (size_t)((a->batch - 1) * a->table_stride + a->table_pages) * 4) ||
        overlap(caches[i], bytes[i], a->lengths, (size_t)a->batch * 4) ||
        overlap(caches[i], bytes[i], a->nodes, (size_t)a->batch * a->tokens * 4) ||
        overlap(caches[i], bytes[i], a->counts, (size_t)a->batch * 4))
      return TF_E_ALIAS;
  }
  const hipError_t err = tf_exl3::launch_cache_append(*a, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? TF_OK : TF_E_LAUNCH;
}

size_t tf_exl3_verify_workspace(int batch, int nodes, int vocab) {
  return verify_sizes(batch, nodes, vocab, false) == TF_OK ? tf_exl3::verify_workspace(batch, nodes, vocab) : 0;
}

int tf_exl3_verify_tree(int dtype, int batch, int nodes, int vocab, const void* logits, int64_t stride_batch,
                        int64_t stride_node, const int32_t* tokens, const int32_t* parents, const float* u,
                        const float* temperature, int32_t* accepted, int32_t* count, int32_t* next,
                        void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return TF_E_DTYPE;
  const int st = verify_sizes(batch, nodes, vocab, true);
  if (st != TF_OK) return st;
  if (!row_strides_ok(stride_batch, stride_node)) return TF_E_SIZE;
  if (batch == 0) return TF_OK;
  if (!logits || !tokens || !parents || !u || !accepted || !count || !next || !workspace) return TF_E_NULL;
  if (!aligned(logits, elem_size(dtype)) || !aligned(tokens, 4) || !aligned(parents, 4) || !aligned(u, 4) ||
      !aligned(temperature, 4) || !aligned(accepted, 4) || !aligned(count, 4) || !aligned(next, 4) ||
      !aligned(workspace, 16))
    return TF_E_ALIGN;
  const size_t need = tf_exl3::verify_workspace(batch, nodes, vocab);
  if (workspace_bytes < need) return TF_E_WORKSPACE;
  const size_t n = (size_t)batch * nodes * 4, nb = (size_t)batch * 4;
  const int64_t s[3] = {stride_batch, stride_node, 0};
  const void* in[5] = {logits, tokens, parents, u, temperature};
  const size_t in_bytes[5] = {extent(batch, nodes, 1, vocab, s, elem_size(dtype)), n, n, n, nb};
  const void* out[4] = {accepted, count, next, workspace};
  const size_t out_bytes[4] = {n, nb, nb, need};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 5; ++i)
      if (overlap(out[o], out_bytes[o], in[i], in_bytes[i])) return TF_E_ALIAS;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out_bytes[o], out[i], out_bytes[i])) return TF_E_ALIAS;
  }
  tf_exl3::VerifyArgs a = {};
  a.dtype = dtype, a.batch = batch, a.nodes = nodes, a.vocab = vocab;
  a.logits = logits, a.stride_batch = stride_batch, a.stride_node = stride_node;
  a.tokens = tokens, a.parents = parents, a.u = u, a.temperature = temperature;
  a.accepted = accepted, a.count = count, a.next = next, a.workspace = workspace;
  const hipError_t e = tf_exl3::launch_verify(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TF_OK : TF_E_LAUNCH;
}

int tf_exl3_verify_chain(int dtype, int batch, int nodes, int vocab, const void* logits, int64_t stride_batch,
                         int64_t stride_node, const int32_t* tokens, const float* q, int64_t q_stride_batch,
                         int64_t q_stride_node, const float* u, const float* temperature, int32_t* count,
                         int32_t* next, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return TF_E_DTYPE;
  const int st = verify_sizes(batch, nodes, vocab, false);
  if (st != TF_OK) return st;
  if (!row_strides_ok(stride_batch, stride_node) || !row_strides_ok(q_stride_batch, q_stride_node)) return TF_E_SIZE;
  if (batch == 0) return TF_OK;
  if (!logits || !tokens || (!q && nodes > 1) || !u || !count || !next || !workspace) return TF_E_NULL;
  if (!aligned(logits, elem_size(dtype)) || !aligned(tokens, 4) || !aligned(q, 4) || !aligned(u, 4) ||
      !aligned(temperature, 4) || !aligned(count, 4) || !aligned(next, 4) || !aligned(workspace, 16))
    return TF_E_ALIGN;
  const size_t need = tf_exl3::verify_workspace(batch, nodes, vocab);
  if (workspace_bytes < need) return TF_E_WORKSPACE;
  const size_t n = (size_t)batch * nodes * 4, nb = (size_t)batch * 4;
  const int64_t s[3] = {stride_batch, stride_node, 0}, sq[3] = {q_stride_batch, q_stride_node, 0};
  const void* in[5] = {logits, tokens, u, temperature, q};
  const size_t in_bytes[5] = {extent(batch, nodes, 1, vocab, s, elem_size(dtype)), n, n, nb,
                              nodes > 1 ? extent(batch, nodes - 1, 1, vocab, sq, 4) : 0};
  const void* out[3] = {count, next, workspace};
  const size_t out_bytes[3] = {nb, nb, need};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 5; ++i)
      if (overlap(out[o], out_bytes[o], in[i], in_bytes[i])) return TF_E_ALIAS;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out_bytes[o], out[i], out_bytes[i])) return TF_E_ALIAS;
  }
  tf_exl3::VerifyArgs a = {};
  a.dtype = dtype, a.batch = batch, a.nodes = nodes, a.vocab = vocab;
  a.logits = logits, a.stride_batch = stride_batch, a.stride_node = stride_node;
  a.tokens = tokens, a.q = q, a.q_stride_batch = q_stride_batch, a.q_stride_node = q_stride_node;
  a.u = u, a.temperature = temperature, a.count = count, a.next = next, a.workspace = workspace;
  const hipError_t e = tf_exl3::launch_verify(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? TF_OK : TF_E_LAUNCH;
}

size_t tf_exl3_distill_workspace(int dtype, int rows, int vocab, int top_k) {
  if (!dtype_ok(dtype) || rows < 0 || vocab < 1 || top_k < 1 || top_k > kMaxTop || !tf_exl3::distill_fits(dtype, rows, vocab))
    return 0;
  return tf_exl3::distill_workspace(dtype, rows, vocab, top_k);
}

int tf_exl3_distill(int dtype, int rows, int vocab, int top_k, const void* logits, int64_t logits_stride,
                    const int32_t* index, const void* top, int top_dtype, const float* weight, float temperature,
                    float* loss, void* grad, int64_t grad_stride, void* workspace, size_t workspace_bytes,
                    void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(top_dtype)) return TF_E_DTYPE;
  if (rows < 0 || vocab < 1 || top_k < 1 || top_k > kMaxTop || !tf_exl3::distill_fits(dtype, rows, vocab)) return TF_E_SIZE;
  if (!(temperature > 0.f) || !isfinite(temperature) || !isfinite(1.f / temperature)) return TF_E_SIZE;
  if (logits_stride < 0 || logits_stride > kMaxStride) return TF_E_SIZE;
  if (grad && (grad_stride < 0 || grad_stride > kMaxStride || (rows > 1 && grad_stride < vocab))) return TF_E_SIZE;
  if (rows == 0) return TF_OK;
  if (!logits || !index || !top || (!loss && !grad) || (grad && !weight) || !workspace) return TF_E_NULL;
  const size_t e = elem_size(dtype);
  if (!aligned(logits, e) || !aligned(grad, e) || !aligned(index, 4) || !aligned(top, elem_size(top_dtype)) ||
      !aligned(weight, 4) || !aligned(loss, 4) || !aligned(workspace, 16))
    return TF_E_ALIGN;
  const size_t need = tf_exl3::distill_workspace(dtype, rows, vocab, top_k);
  if (workspace_bytes < need) return TF_E_WORKSPACE;
  const size_t entries = (size_t)rows * top_k;
  const void* in[4] = {logits, index, top, grad ? weight : nullptr};
  const size_t in_bytes[4] = {(size_t)((rows - 1) * logits_stride + vocab) * e, entries * 4,
                              entries * elem_size(top_dtype), (size_t)rows * 4};
  const void* out[3] = {loss, grad, workspace};
  const size_t out_bytes[3] = {(size_t)rows * 4, (size_t)((rows - 1) * grad_stride + vocab) * e, need};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 4; ++i)
      if (overlap(out[o], out_bytes[o], in[i], in_bytes[i])) return TF_E_ALIAS;
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out_bytes[o], out[i], out_bytes[i])) return TF_E_ALIAS;
  }
  tf_exl3::DistillArgs a = {};
  a.dtype = dtype, a.rows = rows, a.vocab = vocab, a.top_k = top_k;
  a.logits = logits, a.logits_stride = logits_stride, a.index = index, a.top = top, a.top_dtype = top_dtype;
  a.weight = weight, a.temperature = temperature, a.loss = loss, a.grad = grad, a.grad_stride = grad_stride;
  a.workspace = workspace;
  const hipError_t err = tf_exl3::launch_distill(a, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? TF_OK : TF_E_LAUNCH;
}

}  // extern "C"
