// Host side of the attention over the paged cache: workspace, tensor maps,
// choice of kernels.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn.cuh"

namespace lora {

cudaError_t launch_attn_decode(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                               const AttnParams& P, cudaStream_t st, const DeviceInfo& dev);
cudaError_t launch_attn_prefill(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                const CUtensorMap& tm_v, const AttnParams& P, cudaStream_t st,
                                const DeviceInfo& dev);

namespace {

// The kernel of a phase, by the rows of a key head that the longest run of
// new tokens has: up to 16 the keys stand in the MMA's M and the rows (4, 8 or
// 16 of them) in N; above, the rows stand in M, in two halves of whole tokens.
// Measured with 24 rows on ~3000 keys (8 key heads of 128), rows in N with room
// for 32 against rows in M: 1 sequence 25.7 : 19.8 us, 8 sequences 36.2 : 33.1
// us, 64 sequences 137.7 : 141.1 us; with 40 rows 24.6 : 20.2, 47.2 : 32.0 and
// 242.8 : 135.2 us.  (A key head of more than 128 query heads does not fit a
// half: its rows are cut into tiles of 16.)
struct Shape {
  bool prefill;
  int rows;   // of a row tile
  int space;  // rows that a part of one has room for
};
Shape shape_of(int64_t tokens, int group) {
  const int64_t rows = (tokens > 1 ? tokens : 1) * group;
  if (rows > 16 && group <= 128) return {true, 2 * (128 / group) * group, 256};
  const int n = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
  return {false, n, n};
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// The workspace: the error word, the counters (at one place for all batches, so
// that batches can share a workspace), then what one call writes and reads.
struct Layout {
  size_t count, split, part, part_ml, prior, prior_lse, bytes;
  Shape shape[2];  // sequences, groups
};

Layout layout(const lora_paged_kv_t& kv, int n_q_heads, int n_groups) {
  Layout w;
  const int group = n_q_heads / kv.n_kv_heads;
  w.shape[0] = shape_of(kv.max_q_len < kv.T ? kv.max_q_len : kv.T, group);
  w.shape[1] = shape_of(kv.T, group);
  int space = w.shape[0].space;
  if (n_groups > 0 && w.shape[1].space > space) space = w.shape[1].space;
  const size_t slots = static_cast<size_t>(kDecodeScheduleCtas) * 2 * space;
  w.count = 256;
  w.split = up256(w.count + kDecodeScheduleCtas * 2 * sizeof(uint32_t));
  w.part = up256(w.split + kDecodeScheduleCtas * sizeof(SplitItem));
  w.part_ml = w.part + slots * kv.head_dim * 4;
  w.prior = up256(w.part_ml + slots * 8);
  const size_t rows_all = n_groups > 0 ? static_cast<size_t>(kv.T) * n_q_heads : 0;
  w.prior_lse = w.prior + rows_all * kv.head_dim * 4;
  w.bytes = up256(w.prior_lse + rows_all * 4);
  return w;
}

// One cache as [groups of 8 rows][64-value halves of a head][8 rows][64
// values], the order in which a box lands in shared memory: eight rows of 128
// bytes are one atom of the 128-byte swizzle, the halves of a head are
// neighbours, pages and boxes of any height follow one another evenly.
bool encode_cache_map(CUtensorMap* m, void* base, const lora_paged_kv_t& kv) {
  const uint64_t d = kv.head_dim;
  const uint64_t groups =
      static_cast<uint64_t>(kv.n_pages) * kv.n_kv_heads * (kv.page_size / 8);
  const uint64_t dims[4] = {64, 8, d / 64, groups};
  const uint64_t strides[3] = {d * 2, 128, d * 16};
  const uint32_t box[4] = {64, 8, static_cast<uint32_t>(d / 64),
                           static_cast<uint32_t>((kv.page_size < kKeys ? kv.page_size : kKeys) / 8)};
  return encode_tensor_map_bf16_4d(m, base, dims, strides, box);
}

// q as [64-value halves][tokens][heads][64 values]: a box is whole tokens' query
// heads of one key head, rows of 128 bytes.
bool encode_q_map(CUtensorMap* m, const AttnArgs& a, const lora_paged_kv_t& kv, int group) {
  const uint64_t d = kv.head_dim;
  const uint64_t dims[4] = {64, static_cast<uint64_t>(a.n_q_heads), static_cast<uint64_t>(kv.T),
                            d / 64};
  const uint64_t strides[3] = {d * 2, static_cast<uint64_t>(a.q_stride) * 2, 128};
  const uint32_t box[4] = {64, static_cast<uint32_t>(group), static_cast<uint32_t>(128 / group), 1};
  return encode_tensor_map_bf16_4d(m, a.q, dims, strides, box);
}

}  // namespace

size_t attn_ws_bytes(const lora_paged_kv_t& kv, int n_q_heads, int n_groups) {
  return layout(kv, n_q_heads, n_groups).bytes;
}

cudaError_t launch_attn(const lora_paged_kv_t& kv, const AttnArgs& a, cudaStream_t st,
                        const DeviceInfo& dev) {
  CUtensorMap tm_q, tm_k, tm_v;
  if (!encode_cache_map(&tm_k, kv.k_cache, kv) || !encode_cache_map(&tm_v, kv.v_cache, kv))
    return cudaErrorInvalidValue;
  const Layout w = layout(kv, a.n_q_heads, a.n_groups);
  uint8_t* base = static_cast<uint8_t*>(a.ws);
  AttnParams P = {};
  P.kv = kv;
  P.q = static_cast<const bf16*>(a.q);
  P.q_stride = a.q_stride;
  P.out = static_cast<bf16*>(a.out);
  P.out_stride = a.out_stride;
  P.group_off = a.group_off;
  P.prefix_len = a.prefix_len;
  P.n_groups = a.n_groups;
  P.group = a.n_q_heads / kv.n_kv_heads;
  P.by_group = FastDiv::of(P.group);
  P.n_q_heads = a.n_q_heads;
  P.lg_page = 31 - __builtin_clz(static_cast<unsigned>(kv.page_size));
  P.box = kv.page_size < kKeys ? kv.page_size : kKeys;
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.window = a.window;
  P.n_sink = a.n_sink;
  P.err = static_cast<uint32_t*>(a.ws);
  P.count = reinterpret_cast<uint32_t*>(base + w.count);
  P.split = reinterpret_cast<SplitItem*>(base + w.split);
  P.part = reinterpret_cast<float*>(base + w.part);
  P.part_ml = reinterpret_cast<float*>(base + w.part_ml);
  P.prior = reinterpret_cast<float*>(base + w.prior);
  P.prior_lse = reinterpret_cast<float*>(base + w.prior_lse);
  for (int phase = a.n_groups > 0 ? 1 : 0; phase >= 0; --phase) {
    P.groups_phase = phase == 1;
    P.rows = w.shape[phase].rows;
    P.by_rows = FastDiv::of(P.rows);
    // Beside its key tiles an item costs its first scores and its results: in the
    // prefill kernel as much as three tiles (prompt of 8192: 346 us; 2, 4 and 5
    // units 352, 349 and 355), in the other, where a second warpgroup is at work, one.
    // Splitting an item costs each of its CTAs a part, so short ones stay whole:
    // up to 8 tiles of single tokens (the tokens after a prefix of 8K: 56.5 us,
    // split 59.8), two of prompts.
    P.over = w.shape[phase].prefill ? 3 : 1;
    P.whole = w.shape[phase].prefill ? 2 : 8;
    // By the fewest items that this many rows can make: with 38 and more one has
    // a few parts, which the last CTA to arrive adds up; fewer items have many
    // parts, 128 KB each, more than one SM reads in good time.  In the kernel
    // against by a kernel of its own: prompt of 4096 (512 items) 123.5 : 141.1 us,
    // 60 rows on 30000 (8 items) 65.4 : 41.7 us, prefix of 8K (8 items) 70.7 :
    // 50.6 us.
    P.join_after = static_cast<int64_t>(kv.T) * P.group / P.rows * kv.n_kv_heads < 38;
    cudaError_t e;
    if (w.shape[phase].prefill) {
      if (!encode_q_map(&tm_q, a, kv, P.group)) return cudaErrorInvalidValue;
      e = launch_attn_prefill(tm_q, tm_k, tm_v, P, st, dev);
    } else {
      e = launch_attn_decode(tm_k, tm_v, P, st, dev);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace lora
