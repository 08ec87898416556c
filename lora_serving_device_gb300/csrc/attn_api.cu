// C-ABI entry points of the paged-cache operators (declared in
// include/lora.h): argument validation and kernel enqueueing.  Nothing here
// allocates device memory or synchronises.
#include "attn.h"

namespace lora {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool page_size_ok(int pg) { return pg >= 8 && pg <= 256 && (pg & (pg - 1)) == 0; }

bool kv_shape_ok(const lora_paged_kv_t& kv) {
  const int pg = kv.page_size;
  return kv.T <= LORA_MAX_TOKENS && kv.n_seqs >= 1 && kv.n_seqs <= LORA_MAX_SEQS &&
         kv.n_pages >= 1 && kv.max_pages >= 1 && page_size_ok(pg) &&
         (kv.head_dim == 64 || kv.head_dim == 128) && kv.n_kv_heads >= 1 &&
         kv.n_kv_heads <= LORA_MAX_HEADS &&
         // positions, and what the kernels round up from them (tiles, pages), in 32 bits
         static_cast<int64_t>(kv.max_pages) * pg <= INT32_MAX - 1023 &&
         // eight-row groups of one cache, the tensor map's outermost extent
         static_cast<int64_t>(kv.n_pages) * kv.n_kv_heads * (pg / 8) <= INT32_MAX;
}

lora_status_t check_kv(const lora_paged_kv_t* kv) {
  if (kv == nullptr || kv->T < 0 || kv->n_seqs < 0 || kv->n_pages < 0 || kv->max_q_len < 0)
    return LORA_ERR_INVALID_ARG;
  if (!kv_shape_ok(*kv)) return LORA_ERR_SHAPE;
  if (kv->k_cache == nullptr || kv->v_cache == nullptr || kv->block_table == nullptr ||
      kv->q_off == nullptr || kv->kv_len == nullptr || !aligned16(kv->k_cache) ||
      !aligned16(kv->v_cache) || !aligned4(kv->block_table) || !aligned4(kv->q_off) ||
      !aligned4(kv->kv_len))
    return LORA_ERR_INVALID_ARG;
  return LORA_OK;
}

// Rows [T, heads, head_dim]: 16-byte loads from every head of every row, and
// rows that do not overlap.  An empty batch has no rows to point to.
lora_status_t check_rows(const void* p, int64_t stride, const lora_paged_kv_t& kv, int heads) {
  if ((p == nullptr && kv.T > 0) || !aligned16(p)) return LORA_ERR_INVALID_ARG;
  if (stride % 8 != 0 || stride > (int64_t{1} << 38) ||
      stride < static_cast<int64_t>(heads) * kv.head_dim)
    return LORA_ERR_SHAPE;
  return LORA_OK;
}

bool q_heads_ok(int n_q, const lora_paged_kv_t& kv) {
  return n_q >= 1 && n_q <= LORA_MAX_HEADS && n_q % kv.n_kv_heads == 0;
}

lora_status_t check_ws(const void* ws, size_t bytes, size_t need) {
  return ws == nullptr || !aligned16(ws) || bytes < need ? LORA_ERR_WORKSPACE : LORA_OK;
}

lora_status_t check_scales(const uint8_t* k, const uint8_t* v) {
  return k == nullptr || v == nullptr || !aligned16(k) || !aligned16(v) ? LORA_ERR_INVALID_ARG
                                                                         : LORA_OK;
}

lora_status_t attn_common(const lora_paged_kv_t* kv, const AttnArgs& a, bool bits8,
                          size_t ws_bytes, void* stream) {
  lora_status_t s = check_kv(kv);
  if (s != LORA_OK) return s;
  if (!q_heads_ok(a.n_q_heads, *kv)) return LORA_ERR_SHAPE;
  if ((s = check_rows(a.q, a.q_stride, *kv, a.n_q_heads)) != LORA_OK) return s;
  if ((s = check_rows(a.out, a.out_stride, *kv, a.n_q_heads)) != LORA_OK) return s;
  if (bits8 && (s = check_scales(a.k_scale, a.v_scale)) != LORA_OK) return s;
  if ((a.q == a.out && a.q != nullptr) || !(a.scale > 0.f && a.scale < 1e30f) || a.window < 0 || a.n_sink < 0)
    return LORA_ERR_INVALID_ARG;
  if ((s = check_ws(a.ws, ws_bytes, attn_ws_bytes(*kv, a.n_q_heads, a.n_groups))) != LORA_OK)
    return s;
  if (kv->T == 0) return LORA_OK;
  DeviceInfo dev;
  if ((s = check_device(&dev)) != LORA_OK) return s;
  return launch_attn(*kv, a, static_cast<cudaStream_t>(stream), dev) == cudaSuccess
             ? LORA_OK
             : LORA_ERR_CUDA;
}

lora_status_t append_common(const lora_paged_kv_t* kv, bool bits8, uint8_t* k_scale,
                            uint8_t* v_scale, const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, const void* v, int64_t v_stride, int32_t n_q_heads,
                            const float* cos_sin, int32_t n_pos, int32_t rot_dim,
                            const int32_t* pos, int32_t n_axes, const int32_t* axis_pairs,
                            int32_t interleaved, void* q_out, int64_t q_out_stride, void* ws,
                            size_t ws_bytes, void* stream) {
  lora_status_t s = check_kv(kv);
  if (s != LORA_OK) return s;
  if (rot_dim < 0 || rot_dim % 16 != 0 || rot_dim > kv->head_dim || n_axes < 1 ||
      n_axes > LORA_MAX_POS_AXES || n_pos < 0 ||
      (n_q_heads != 0 && !q_heads_ok(n_q_heads, *kv)))
    return LORA_ERR_SHAPE;
  AppendArgs a = {};
  if (rot_dim > 0 && (cos_sin == nullptr || !aligned16(cos_sin) || n_pos < 1))
    return LORA_ERR_INVALID_ARG;
  if (n_axes > 1) {
    if ((pos == nullptr && kv->T > 0) || axis_pairs == nullptr) return LORA_ERR_INVALID_ARG;
    int64_t sum = 0;
    for (int i = 0; i < n_axes; ++i) {
      if (axis_pairs[i] < 0) return LORA_ERR_INVALID_ARG;
      sum += axis_pairs[i];
      if (sum > rot_dim / 2) return LORA_ERR_SHAPE;
      a.axis_end[i] = static_cast<int>(sum);
    }
    if (sum != rot_dim / 2) return LORA_ERR_SHAPE;
  } else {
    if (axis_pairs != nullptr && axis_pairs[0] != rot_dim / 2) return LORA_ERR_SHAPE;
    a.axis_end[0] = rot_dim / 2;
  }
  for (int i = n_axes; i < LORA_MAX_POS_AXES; ++i) a.axis_end[i] = rot_dim / 2;
  if (!aligned4(pos)) return LORA_ERR_INVALID_ARG;
  if ((s = check_rows(k, k_stride, *kv, kv->n_kv_heads)) != LORA_OK) return s;
  if ((s = check_rows(v, v_stride, *kv, kv->n_kv_heads)) != LORA_OK) return s;
  if (n_q_heads > 0) {
    if ((s = check_rows(q, q_stride, *kv, n_q_heads)) != LORA_OK) return s;
    if ((s = check_rows(q_out, q_out_stride, *kv, n_q_heads)) != LORA_OK) return s;
    if (q == q_out && q_stride != q_out_stride) return LORA_ERR_INVALID_ARG;
  }
  if (bits8 && (s = check_scales(k_scale, v_scale)) != LORA_OK) return s;
  if ((s = check_ws(ws, ws_bytes, 16)) != LORA_OK) return s;
  if (kv->T == 0) return LORA_OK;
  DeviceInfo dev;
  if ((s = check_device(&dev)) != LORA_OK) return s;
  a.q = q, a.k = k, a.v = v;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.n_q_heads = n_q_heads;
  a.cos_sin = cos_sin, a.n_pos = n_pos, a.rot_dim = rot_dim;
  a.pos = pos, a.n_axes = n_axes, a.interleaved = interleaved;
  a.q_out = q_out, a.q_out_stride = q_out_stride;
  a.err = static_cast<uint32_t*>(ws);
  a.k_scale = k_scale, a.v_scale = v_scale;
  const auto st = static_cast<cudaStream_t>(stream);
  return (bits8 ? launch_kv_append_8bit(*kv, a, st) : launch_kv_append(*kv, a, st)) == cudaSuccess
             ? LORA_OK
             : LORA_ERR_CUDA;
}

lora_status_t prefix_common(const lora_paged_kv_t* kv, const AttnArgs& a, bool bits8,
                            size_t ws_bytes, void* stream) {
  const lora_status_t s = check_kv(kv);
  if (s != LORA_OK) return s;
  if (a.n_groups < 1 || a.n_groups > kv->n_seqs) return LORA_ERR_SHAPE;
  if (a.group_off == nullptr || a.prefix_len == nullptr || !aligned4(a.group_off) ||
      !aligned4(a.prefix_len))
    return LORA_ERR_INVALID_ARG;
  return attn_common(kv, a, bits8, ws_bytes, stream);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" {

size_t lora_attn_workspace_bytes(const lora_paged_kv_t* kv, int32_t n_q_heads, int32_t n_groups) {
  if (kv == nullptr || kv->T < 0 || !kv_shape_ok(*kv) || !q_heads_ok(n_q_heads, *kv) ||
      n_groups < 0 || n_groups > kv->n_seqs)
    return 16;
  return attn_ws_bytes(*kv, n_q_heads, n_groups);
}

lora_status_t lora_kv_append(const lora_paged_kv_t* kv, const void* q, int64_t q_stride,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             int32_t n_q_heads, const float* cos_sin, int32_t n_pos,
                             int32_t rot_dim, const int32_t* pos, int32_t n_axes,
                             const int32_t* axis_pairs, int32_t interleaved, void* q_out,
                             int64_t q_out_stride, void* ws, size_t ws_bytes, void* stream) {
  return append_common(kv, false, nullptr, nullptr, q, q_stride, k, k_stride, v, v_stride,
                       n_q_heads, cos_sin, n_pos, rot_dim, pos, n_axes, axis_pairs, interleaved,
                       q_out, q_out_stride, ws, ws_bytes, stream);
}

lora_status_t lora_kv_append_8bit(const lora_paged_kv_t* kv, uint8_t* k_scale, uint8_t* v_scale,
                                  const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride,
                                  int32_t n_q_heads, const float* cos_sin, int32_t n_pos,
                                  int32_t rot_dim, const int32_t* pos, int32_t n_axes,
                                  const int32_t* axis_pairs, int32_t interleaved, void* q_out,
                                  int64_t q_out_stride, void* ws, size_t ws_bytes, void* stream) {
  return append_common(kv, true, k_scale, v_scale, q, q_stride, k, k_stride, v, v_stride,
                       n_q_heads, cos_sin, n_pos, rot_dim, pos, n_axes, axis_pairs, interleaved,
                       q_out, q_out_stride, ws, ws_bytes, stream);
}

lora_status_t lora_attn_paged(const lora_paged_kv_t* kv, const void* q, int64_t q_stride,
                              int32_t n_q_heads, float scale, int32_t window, int32_t n_sink,
                              void* out, int64_t out_stride, void* ws, size_t ws_bytes,
                              void* stream) {
  const AttnArgs a = {q, q_stride, n_q_heads, scale, window, n_sink, nullptr, nullptr,
                      0, out,      out_stride, ws,   nullptr, nullptr};
  return attn_common(kv, a, false, ws_bytes, stream);
}

lora_status_t lora_attn_paged_8bit(const lora_paged_kv_t* kv, const uint8_t* k_scale,
                                   const uint8_t* v_scale, const void* q, int64_t q_stride,
                                   int32_t n_q_heads, float scale, int32_t window,
                                   int32_t n_sink, void* out, int64_t out_stride, void* ws,
                                   size_t ws_bytes, void* stream) {
  const AttnArgs a = {q, q_stride, n_q_heads, scale, window, n_sink, nullptr, nullptr,
                      0, out,      out_stride, ws,   k_scale, v_scale};
  return attn_common(kv, a, true, ws_bytes, stream);
}

lora_status_t lora_attn_prefix(const lora_paged_kv_t* kv, const int32_t* group_off,
                               const int32_t* prefix_len, int32_t n_groups, const void* q,
                               int64_t q_stride, int32_t n_q_heads, float scale, void* out,
                               int64_t out_stride, void* ws, size_t ws_bytes, void* stream) {
  const AttnArgs a = {q,         q_stride,   n_q_heads, scale, 0,          0,  group_off,
                      prefix_len, n_groups,  out,       out_stride, ws,    nullptr, nullptr};
  return prefix_common(kv, a, false, ws_bytes, stream);
}

lora_status_t lora_attn_prefix_8bit(const lora_paged_kv_t* kv, const uint8_t* k_scale,
                                    const uint8_t* v_scale, const int32_t* group_off,
                                    const int32_t* prefix_len, int32_t n_groups, const void* q,
                                    int64_t q_stride, int32_t n_q_heads, float scale, void* out,
                                    int64_t out_stride, void* ws, size_t ws_bytes, void* stream) {
  const AttnArgs a = {q,         q_stride,   n_q_heads, scale, 0,          0,  group_off,
                      prefix_len, n_groups,  out,       out_stride, ws,    k_scale, v_scale};
  return prefix_common(kv, a, true, ws_bytes, stream);
}

size_t lora_batch_plan_workspace_bytes(int32_t n_seqs) {
  return n_seqs < 1 || n_seqs > LORA_MAX_SEQS ? 16 : 256 + static_cast<size_t>(n_seqs) * 24;
}

lora_status_t lora_batch_plan(const int32_t* n_cached, const int32_t* n_new,
                              const int32_t* n_shared, int32_t n_seqs, int32_t T,
                              int32_t page_size, int32_t max_pages, int32_t n_pages,
                              int32_t* free_pages, int32_t free_cap, const int32_t* n_free,
                              int32_t* block_table, int32_t* q_off, int32_t* kv_len,
                              int64_t* slots, int32_t* pos, int32_t* n_free_out, void* ws,
                              size_t ws_bytes, void* stream) {
  if (n_seqs < 0 || T < 0 || n_pages < 0) return LORA_ERR_INVALID_ARG;
  if (T > LORA_MAX_TOKENS || n_seqs < 1 || n_seqs > LORA_MAX_SEQS || !page_size_ok(page_size) ||
      max_pages < 1 || n_pages < 1 || free_cap < 1 ||
      // positions and the rows after them, rounded up to pages, in 32 bits
      static_cast<int64_t>(max_pages) * page_size > INT32_MAX - 1023 - T)
    return LORA_ERR_SHAPE;
  for (const int32_t* p : {n_cached, n_new, static_cast<const int32_t*>(free_pages), n_free,
                           static_cast<const int32_t*>(block_table),
                           static_cast<const int32_t*>(q_off), static_cast<const int32_t*>(kv_len),
                           static_cast<const int32_t*>(n_free_out)})
    if (p == nullptr || !aligned4(p)) return LORA_ERR_INVALID_ARG;
  if (!aligned4(n_shared) || !aligned4(pos) || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
    return LORA_ERR_INVALID_ARG;
  const lora_status_t s = check_ws(ws, ws_bytes, lora_batch_plan_workspace_bytes(n_seqs));
  if (s != LORA_OK) return s;
  DeviceInfo dev;
  const lora_status_t d = check_device(&dev);
  if (d != LORA_OK) return d;
  uint8_t* base = static_cast<uint8_t*>(ws);
  PlanArgs a = {};
  a.n_cached = n_cached, a.n_new = n_new, a.n_shared = n_shared;
  a.n_seqs = n_seqs, a.T = T, a.page_size = page_size, a.max_pages = max_pages;
  a.lg_page = 31 - __builtin_clz(static_cast<unsigned>(page_size));
  a.n_pages = n_pages;
  a.free_pages = free_pages, a.free_cap = free_cap, a.n_free = n_free;
  a.block_table = block_table, a.q_off = q_off, a.kv_len = kv_len;
  a.slots = slots, a.pos = pos, a.n_free_out = n_free_out;
  a.err = static_cast<uint32_t*>(ws);
  a.top = reinterpret_cast<int32_t*>(base + 128);
  a.give_off = reinterpret_cast<int64_t*>(base + 256);
  a.take_off = reinterpret_cast<int32_t*>(a.give_off + n_seqs);
  a.give = a.take_off + n_seqs;
  a.span = a.give + n_seqs;
  return launch_batch_plan(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LORA_OK
                                                                                : LORA_ERR_CUDA;
}

}  // extern "C"
