// Internal launch interface between the C ABI of the operators around the projection
// (ops_abi.cpp) and their kernels. Arguments reaching these functions have been checked.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "tf_exl3.h"

namespace tf_exl3 {

// The runtime refuses a launch with 2^32 work-items or more in a dimension. Each operator says
// beforehand whether all launches of a call stay below, so that none is left out behind others.
inline bool launchable(int64_t workgroups, int threads) { return workgroups * threads < (1ll << 32); }

bool tree_attention_fits(const tf_exl3_tree_attention_args& a);
hipError_t launch_tree_attention(const tf_exl3_tree_attention_args& a, hipStream_t stream);
size_t tree_attention_workspace(const tf_exl3_tree_attention_args& a);

// The same with a cache in 4 bits, whose strides are in bytes.
bool tree_attention_q4_fits(const tf_exl3_tree_attention_args& a);
hipError_t launch_tree_attention_q4(const tf_exl3_tree_attention_args& a, hipStream_t stream);
size_t tree_attention_q4_workspace(const tf_exl3_tree_attention_args& a);

bool cache_append_fits(const tf_exl3_cache_append_args& a);
hipError_t launch_cache_append(const tf_exl3_cache_append_args& a, hipStream_t stream);

bool cache_append_q4_fits(const tf_exl3_cache_append_q4_args& a);
hipError_t launch_cache_append_q4(const tf_exl3_cache_append_q4_args& a, hipStream_t stream);
bool cache_read_q4_fits(const tf_exl3_cache_read_q4_args& a);
hipError_t launch_cache_read_q4(const tf_exl3_cache_read_q4_args& a, hipStream_t stream);

hipError_t launch_norm_rotate(const tf_exl3_norm_rotate_args& a, hipStream_t stream);

bool prompt_attention_fits(const tf_exl3_prompt_attention_args& a);
hipError_t launch_prompt_attention(const tf_exl3_prompt_attention_args& a, hipStream_t stream);

struct VerifyArgs {
  int dtype, batch, nodes, vocab;
  const void* logits;
  int64_t stride_batch, stride_node;
  const int32_t* tokens;
  const int32_t* parents;  // the tree's; nullptr for a chain
  const float* q;          // the chain's drafter; nullptr for a tree
  int64_t q_stride_batch, q_stride_node;
  const float* u;
  const float* temperature;
  int32_t *accepted, *count, *next;
  void* workspace;
};

bool verify_fits(int batch, int nodes, int vocab, bool tree);
hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream);
size_t verify_workspace(int batch, int nodes, int vocab);

struct DistillArgs {
  int dtype, rows, vocab, top_k;
  const void* logits;
  int64_t logits_stride;
  const int32_t* index;
  const void* top;
  int top_dtype;
  const float* weight;
  float temperature;
  float inv, c, c_low;  // 1 / T; log2(e) / T in two parts
  float* loss;
  void* grad;
  int64_t grad_stride;
  void* workspace;
};

bool distill_fits(int dtype, int rows, int vocab);
hipError_t launch_distill(const DistillArgs& a, hipStream_t stream);
size_t distill_workspace(int dtype, int rows, int vocab, int top_k);

}  // namespace tf_exl3
