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
};
// see k_kv_append.cu
cudaError_t launch_kv_append(const lora_paged_kv_t& kv, const AppendArgs& a, cudaStream_t st);

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
};
// see k_attn.cu
cudaError_t launch_attn(const lora_paged_kv_t& kv, const AttnArgs& a, cudaStream_t st,
                        const DeviceInfo& dev);
size_t attn_ws_bytes(const lora_paged_kv_t& kv, int n_q_heads, int n_groups);

}  // namespace lora
