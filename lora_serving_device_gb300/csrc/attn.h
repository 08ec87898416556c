// Launchers of the paged-cache kernels (entry points in attn_api.cu), which
// assume validated arguments.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "internal.h"
#include "lora.h"

namespace lora {

struct AppendArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int n_q_heads;
  const float* cos_sin;
  int n_pos, rot_dim;
  const int32_t* pos;
  int n_axes;
  int axis_end[LORA_MAX_POS_AXES];  // pairs of the axes up to and including this one
  int interleaved;
  void* q_out;
  int64_t q_out_stride;
  uint32_t* err;
  uint8_t *k_scale, *v_scale;  // of a cache in 8 bits
};
// see k_kv_append.cu
cudaError_t launch_kv_append(const lora_paged_kv_t& kv, const AppendArgs& a, cudaStream_t st);
// see k_kv_append_8bit.cu
cudaError_t launch_kv_append_8bit(const lora_paged_kv_t& kv, const AppendArgs& a, cudaStream_t st);

struct PlanArgs {
  const int32_t *n_cached, *n_new, *n_shared;
  int n_seqs, T, page_size, lg_page, max_pages, n_pages;
  int32_t* free_pages;
  int free_cap;
  const int32_t* n_free;
  int32_t *block_table, *q_off, *kv_len;
  int64_t* slots;
  int32_t *pos, *n_free_out;
  uint32_t* err;
  int32_t* top;        // pages on the stack before any is taken
  int32_t* take_off;   // [n_seqs] pages that the sequences before take
  // where kernels of their own count and push the ended requests' pages:
  int64_t* give_off;   // [n_seqs] their places on the stack
  int32_t *give, *span;  // [n_seqs] how many, and [n_seqs][2] the entries that hold them
  bool fill_here;      // one kernel does all
  bool apart;
};
// see k_batch_plan.cu
cudaError_t launch_batch_plan(const PlanArgs& a, cudaStream_t st);

struct AttnArgs {
  const void* q;
  int64_t q_stride;
  int n_q_heads;
  float scale;
  int window, n_sink;
  const int32_t *group_off, *prefix_len;  // prefix groups, or null
  int n_groups;
  void* out;
  int64_t out_stride;
  void* ws;
  const uint8_t *k_scale, *v_scale;  // of a cache in 8 bits, or null
};
// see k_attn.cu
cudaError_t launch_attn(const lora_paged_kv_t& kv, const AttnArgs& a, cudaStream_t st,
                        const DeviceInfo& dev);
size_t attn_ws_bytes(const lora_paged_kv_t& kv, int n_q_heads, int n_groups);

}  // namespace lora
