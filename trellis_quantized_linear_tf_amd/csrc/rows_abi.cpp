// C ABI of the operators between the projection's rows and the cache: norm and rotation, attention
// of prompts, the cache in 4 bits. Argument checks on the host, then one call into the launch interface.
// Nothing is launched or written on a refusal.
#include <math.h>

#include "ops_check.hpp"
#include "ops_launch.hpp"

using namespace tf_exl3;

namespace {

constexpr int kMostHeads = 65535;
constexpr int kMostTokens = 1 << 30;

// Whether two sets of rows alternate in one buffer: of each sequence, of each token, or of each token of each sequence
// the one set's part, then the other's, within a step from one to the next that both have.
bool alternate(const void* a, int heads_a, const int64_t* sa, const void* b, int heads_b, const int64_t* sb, int64_t batch,
               int64_t tokens, int64_t dim, int64_t e) {
  if ((uintptr_t)a > (uintptr_t)b) return alternate(b, heads_b, sb, a, heads_a, sa, batch, tokens, dim, e);
  const int64_t between = (int64_t)((uintptr_t)b - (uintptr_t)a);
  // n0 x n1 rows of all heads, a step apart from the next such part.
  auto within = [&](int64_t step, int64_t n0, int64_t n1) {
    const int64_t one = (n0 - 1) * sa[0] + (n1 - 1) * sa[1] + (heads_a - 1) * sa[2] + dim;
    const int64_t other = (n0 - 1) * sb[0] + (n1 - 1) * sb[1] + (heads_b - 1) * sb[2] + dim;
    return between >= one * e && between + other * e <= step * e;
  };
  const bool sequences = batch > 1 && sa[0] == sb[0], each_token = tokens > 1 && sa[1] == sb[1];
  if (sequences && within(sa[0], 1, tokens)) return true;
  if (each_token && within(sa[1], batch, 1)) return true;
  if (!sequences || !each_token) return false;
  return (sa[0] >= tokens * sa[1] && within(sa[1], 1, 1)) || (sa[1] >= batch * sa[0] && within(sa[0], 1, 1));
}

bool q4_dim_ok(int head_dim) { return head_dim >= 32 && head_dim % 32 == 0 && head_dim <= (1 << 24); }

size_t q4_extent(int pages, int page_size, int heads, int head_dim, const int64_t* s) {
  return extent(pages, page_size, heads, q4_bytes(head_dim), s, 1);
}

template <typename ARGS>
int q4_sizes(const ARGS* a) {
  if (!dtype_ok(a->dtype)) return TF_E_DTYPE;
  if (a->batch < 0 || a->batch > kMaxBatch || a->tokens < 0 || a->tokens > kMostTokens || a->kv_heads < 1 ||
      !q4_dim_ok(a->head_dim) || (int64_t)a->kv_heads * a->head_dim > (1 << 24))
    return TF_E_SIZE;
  const int st = cache_sizes(a->pages, a->page_size, a->table_pages, a->table_stride);
  if (st != TF_OK) return st;
  if (!strides_ok(a->k_stride, 1) || !strides_ok(a->v_stride, 1) || !strides_ok(a->k_cache_stride, 4) ||
      !strides_ok(a->v_cache_stride, 4))
    return TF_E_SIZE;
  return TF_OK;
}

template <typename ARGS>
void q4_settle(ARGS* a) {
  settle(a->batch, a->tokens, a->kv_heads, a->k_stride);
  settle(a->batch, a->tokens, a->kv_heads, a->v_stride);
  settle(a->pages, a->page_size, a->kv_heads, a->k_cache_stride);
  settle(a->pages, a->page_size, a->kv_heads, a->v_cache_stride);
}

size_t table_extent(int batch, int table_pages, int64_t table_stride) {
  return table_pages > 0 ? (size_t)((batch - 1) * table_stride + table_pages) * 4 : 0;
}

}  // namespace

extern "C" {

int tf_exl3_norm_rotate(const tf_exl3_norm_rotate_args* args, void* stream) {
  if (args == nullptr) return TF_E_NULL;
  tf_exl3_norm_rotate_args settled = *args;
  tf_exl3_norm_rotate_args* a = &settled;
  settle(a->batch, a->tokens, a->q_heads, a->q_stride);
  settle(a->batch, a->tokens, a->q_heads, a->q_out_stride);
  settle(a->batch, a->tokens, a->kv_heads, a->k_stride);
  settle(a->batch, a->tokens, a->kv_heads, a->k_out_stride);
  const bool weights = a->norm && (a->q_weight || a->k_weight);
  if (!dtype_ok(a->dtype) || (weights && !dtype_ok(a->weight_dtype))) return TF_E_DTYPE;
  if (a->batch < 0 || a->tokens < 0 || (int64_t)a->batch * a->tokens >= (1 << 24)) return TF_E_SIZE;
  if (a->q_heads < 1 || a->kv_heads < 1 || a->q_heads > kMostHeads || a->kv_heads > kMostHeads) return TF_E_SIZE;
  if (a->head_dim < 16 || a->head_dim > 512 || a->head_dim % 16 != 0) return TF_E_SIZE;
  if (a->rotary_dim != 0 && (a->rotary_dim < 16 || a->rotary_dim > a->head_dim || a->rotary_dim % 8 != 0)) return TF_E_SIZE;
  if (a->norm && !(a->eps >= 0.f && isfinite(a->eps))) return TF_E_SIZE;
  if (a->positions_stride < 0 || a->positions_stride > kMaxStride) return TF_E_SIZE;
  if (!strides_ok(a->q_stride, 1) || !strides_ok(a->k_stride, 1) || !strides_ok(a->q_out_stride, 1) ||
      !strides_ok(a->k_out_stride, 1) || !apart(a->batch, a->tokens, a->q_heads, a->q_out_stride) ||
      !apart(a->batch, a->tokens, a->kv_heads, a->k_out_stride))
    return TF_E_SIZE;
  for (int i = 0; i < 3; ++i)
    if (a->q_stride[i] >= (1ll << 32) || a->k_stride[i] >= (1ll << 32) || a->q_out_stride[i] >= (1ll << 32) ||
        a->k_out_stride[i] >= (1ll << 32))
      return TF_E_SIZE;
  if (a->batch == 0 || a->tokens == 0) return TF_OK;
  if (!a->q || !a->k || !a->q_out || !a->k_out || (a->rotary_dim > 0 && (!a->positions || !a->frequencies))) return TF_E_NULL;
  const size_t e = elem_size(a->dtype), we = elem_size(a->weight_dtype);
  if (!aligned(a->q, e) || !aligned(a->k, e) || !aligned(a->q_out, e) || !aligned(a->k_out, e) || !aligned(a->positions, 4) ||
      !aligned(a->frequencies, 4) || (weights && (!aligned(a->q_weight, we) || !aligned(a->k_weight, we))))
    return TF_E_ALIGN;
  struct Rows {
    const void* p;
    int heads;
    const int64_t* s;
    size_t n;
  };
  auto rows = [&](const void* p, int heads, const int64_t* s) {
    return Rows{p, heads, s, extent(a->batch, a->tokens, heads, a->head_dim, s, e)};
  };
  const Rows in[2] = {rows(a->q, a->q_heads, a->q_stride), rows(a->k, a->kv_heads, a->k_stride)};
  const Rows out[2] = {rows(a->q_out, a->q_heads, a->q_out_stride), rows(a->k_out, a->kv_heads, a->k_out_stride)};
  auto meet = [&](const Rows& x, const Rows& y) {
    return overlap(x.p, x.n, y.p, y.n) &&
           !alternate(x.p, x.heads, x.s, y.p, y.heads, y.s, a->batch, a->tokens, a->head_dim, (int64_t)e);
  };
  for (int o = 0; o < 2; ++o) {
    for (int i = 0; i < 2; ++i) {
      const bool itself = o == i && out[o].p == in[i].p && out[o].s[0] == in[i].s[0] && out[o].s[1] == in[i].s[1] &&
                          out[o].s[2] == in[i].s[2];
      if (!itself && meet(out[o], in[i])) return TF_E_ALIAS;
    }
    const size_t weight = weights ? (size_t)a->head_dim * we : 0;
    if (overlap(out[o].p, out[o].n, a->q_weight, weight) || overlap(out[o].p, out[o].n, a->k_weight, weight) ||
        overlap(out[o].p, out[o].n, a->positions,
                a->rotary_dim > 0 ? (size_t)((a->batch - 1) * a->positions_stride + a->tokens) * 4 : 0) ||
        overlap(out[o].p, out[o].n, a->frequencies, (size_t)a->rotary_dim * 2))
      return TF_E_ALIAS;
  }
  if (meet(out[0], out[1])) return TF_E_ALIAS;
  const hipError_t err = launch_norm_rotate(*a, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? TF_OK : TF_E_LAUNCH;
}

int tf_exl3_prompt_attention(const tf_exl3_prompt_attention_args* args, void* stream) {
  if (args == nullptr) return TF_E_NULL;
  tf_exl3_prompt_attention_args settled = *args;
  tf_exl3_prompt_attention_args* a = &settled;
  if (a->dtype != TF_DT_F16 && a->dtype != TF_DT_BF16) return TF_E_DTYPE;
  if (a->tokens < 0 || a->tokens >= kMostTokens || a->batch < 0 || a->batch >= kMostTokens) return TF_E_SIZE;
  if (a->kv_heads < 1 || a->q_heads < 1 || a->q_heads > kMostHeads || a->q_heads % a->kv_heads != 0) return TF_E_SIZE;
  if (a->head_dim < 16 || a->head_dim > 256 || a->head_dim % 16 != 0) return TF_E_SIZE;
  if (!isfinite(a->scale)) return TF_E_SIZE;
  // Strides of [token, head] as of one sequence.
  int64_t q[3] = {0, a->q_stride[0], a->q_stride[1]}, k[3] = {0, a->k_stride[0], a->k_stride[1]};
  int64_t v[3] = {0, a->v_stride[0], a->v_stride[1]}, o[3] = {0, a->out_stride[0], a->out_stride[1]};
  settle(1, a->tokens, a->q_heads, q);
  settle(1, a->tokens, a->kv_heads, k);
  settle(1, a->tokens, a->kv_heads, v);
  settle(1, a->tokens, a->q_heads, o);
  if (q[1] > (1ll << 31) || o[1] > (1ll << 31)) return TF_E_SIZE;
  if (!strides_ok(q, 8) || !strides_ok(k, 8) || !strides_ok(v, 8) || !strides_ok(o, 4) || !apart(1, a->tokens, a->q_heads, o) ||
      k[1] > (1 << 23) || v[1] > (1 << 23))
    return TF_E_SIZE;
  for (int i = 0; i < 2; ++i)
    a->q_stride[i] = q[i + 1], a->k_stride[i] = k[i + 1], a->v_stride[i] = v[i + 1], a->out_stride[i] = o[i + 1];
  if (!prompt_attention_fits(*a)) return TF_E_SIZE;
  if (a->tokens == 0 || a->batch == 0) return TF_OK;
  if (!a->q || !a->k || !a->v || !a->offsets || !a->out) return TF_E_NULL;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->out, 8) || !aligned(a->offsets, 4))
    return TF_E_ALIGN;
  const size_t no = extent(1, a->tokens, a->q_heads, a->head_dim, o, 2);
  if (overlap(a->out, no, a->q, extent(1, a->tokens, a->q_heads, a->head_dim, q, 2)) ||
      overlap(a->out, no, a->k, extent(1, a->tokens, a->kv_heads, a->head_dim, k, 2)) ||
      overlap(a->out, no, a->v, extent(1, a->tokens, a->kv_heads, a->head_dim, v, 2)) ||
      overlap(a->out, no, a->offsets, ((size_t)a->batch + 1) * 4))
    return TF_E_ALIAS;
  const hipError_t err = launch_prompt_attention(*a, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? TF_OK : TF_E_LAUNCH;
}

size_t tf_exl3_q4_row_bytes(int head_dim) { return q4_dim_ok(head_dim) ? (size_t)q4_bytes(head_dim) : 0; }

int tf_exl3_cache_append_q4(const tf_exl3_cache_append_q4_args* args, void* stream) {
  if (args == nullptr) return TF_E_NULL;
  tf_exl3_cache_append_q4_args settled = *args;
  tf_exl3_cache_append_q4_args* a = &settled;
  q4_settle(a);
  const int st = q4_sizes(a);
  if (st != TF_OK) return st;
  if (!apart(a->pages, a->page_size, a->kv_heads, a->k_cache_stride) || !apart(a->pages, a->page_size, a->kv_heads, a->v_cache_stride))
    return TF_E_SIZE;
  if (a->batch == 0 || a->tokens == 0 || a->table_pages == 0) return TF_OK;
  if (!cache_append_q4_fits(*a)) return TF_E_SIZE;
  if (!a->k || !a->v || !a->k_cache || !a->v_cache || !a->table || !a->lengths) return TF_E_NULL;
  const size_t e = elem_size(a->dtype);
  if (!aligned(a->k, e) || !aligned(a->v, e) || !aligned(a->k_cache, 4) || !aligned(a->v_cache, 4) || !aligned(a->table, 4) ||
      !aligned(a->lengths, 4) || !aligned(a->nodes, 4) || !aligned(a->counts, 4))
    return TF_E_ALIGN;
  const size_t nk = extent(a->batch, a->tokens, a->kv_heads, a->head_dim, a->k_stride, e);
  const size_t nv = extent(a->batch, a->tokens, a->kv_heads, a->head_dim, a->v_stride, e);
  const void* caches[2] = {a->k_cache, a->v_cache};
  const size_t bytes[2] = {q4_extent(a->pages, a->page_size, a->kv_heads, a->head_dim, a->k_cache_stride),
                           q4_extent(a->pages, a->page_size, a->kv_heads, a->head_dim, a->v_cache_stride)};
  for (int i = 0; i < 2; ++i) {
    if (overlap(caches[i], bytes[i], a->k, nk) || overlap(caches[i], bytes[i], a->v, nv) ||
        overlap(caches[i], bytes[i], a->table, table_extent(a->batch, a->table_pages, a->table_stride)) ||
        overlap(caches[i], bytes[i], a->lengths, (size_t)a->batch * 4) ||
        overlap(caches[i], bytes[i], a->nodes, (size_t)a->batch * a->tokens * 4) ||
        overlap(caches[i], bytes[i], a->counts, (size_t)a->batch * 4))
      return TF_E_ALIAS;
  }
  const hipError_t err = launch_cache_append_q4(*a, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? TF_OK : TF_E_LAUNCH;
}

int tf_exl3_cache_read_q4(const tf_exl3_cache_read_q4_args* args, void* stream) {
  if (args == nullptr) return TF_E_NULL;
  tf_exl3_cache_read_q4_args settled = *args;
  tf_exl3_cache_read_q4_args* a = &settled;
  q4_settle(a);
  const int st = q4_sizes(a);
  if (st != TF_OK) return st;
  if (!apart(a->batch, a->tokens, a->kv_heads, a->k_stride) || !apart(a->batch, a->tokens, a->kv_heads, a->v_stride))
    return TF_E_SIZE;
  if (a->batch == 0 || a->tokens == 0) return TF_OK;
  if (!cache_read_q4_fits(*a)) return TF_E_SIZE;
  if (!a->k || !a->v || !a->k_cache || !a->v_cache || !a->lengths || (a->table_pages > 0 && !a->table)) return TF_E_NULL;
  const size_t e = elem_size(a->dtype);
  if (!aligned(a->k, e) || !aligned(a->v, e) || !aligned(a->k_cache, 4) || !aligned(a->v_cache, 4) || !aligned(a->table, 4) ||
      !aligned(a->lengths, 4) || !aligned(a->first, 4))
    return TF_E_ALIGN;
  const void* outs[2] = {a->k, a->v};
  const size_t bytes[2] = {extent(a->batch, a->tokens, a->kv_heads, a->head_dim, a->k_stride, e),
                           extent(a->batch, a->tokens, a->kv_heads, a->head_dim, a->v_stride, e)};
  for (int i = 0; i < 2; ++i) {
    if (overlap(outs[i], bytes[i], a->k_cache, q4_extent(a->pages, a->page_size, a->kv_heads, a->head_dim, a->k_cache_stride)) ||
        overlap(outs[i], bytes[i], a->v_cache, q4_extent(a->pages, a->page_size, a->kv_heads, a->head_dim, a->v_cache_stride)) ||
        overlap(outs[i], bytes[i], a->table, table_extent(a->batch, a->table_pages, a->table_stride)) ||
        overlap(outs[i], bytes[i], a->lengths, (size_t)a->batch * 4) || overlap(outs[i], bytes[i], a->first, (size_t)a->batch * 4))
      return TF_E_ALIAS;
  }
  if (overlap(a->k, bytes[0], a->v, bytes[1])) return TF_E_ALIAS;
  const hipError_t err = launch_cache_read_q4(*a, static_cast<hipStream_t>(stream));
  return err == hipSuccess ? TF_OK : TF_E_LAUNCH;
}

}  // extern "C"
