// Attention over the paged cache (lora_attn_paged, lora_attn_prefix), one
// warp to a (row, query head): the lanes hold head_dim / 32 values of q and
// of the accumulator, keys are taken one by one, the softmax runs along with
// a running maximum and sum.  The definition, executed.
#include "attn.cuh"

namespace lora {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(const lora_paged_kv_t kv,
                                                           const AttnArgs a, uint32_t* err) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / a.n_q_heads), h = static_cast<int>(w % a.n_q_heads);
  if (t >= kv.T) return;
  const int s = seq_of_row(kv.q_off, kv.n_seqs, t);
  if (s < 0) return;
  const int hk = h / (a.n_q_heads / kv.n_kv_heads);
  const int64_t cap = static_cast<int64_t>(kv.max_pages) * kv.page_size;
  int p = kv.kv_len[s] - kv.q_off[s + 1] + t;
  if (p >= cap) {
    flag_error(err, LORA_DEVERR_BAD_LEN);
    p = static_cast<int>(cap) - 1;
  }
  int shared_row = s, shared = 0;
  if (a.group_off != nullptr) {
    int g = seq_of_row(a.group_off, a.n_groups, s);
    if (g >= 0) {
      const int before = kv.kv_len[s] - (kv.q_off[s + 1] - kv.q_off[s]);
      shared = a.prefix_len[g];
      shared_row = a.group_off[g];
      if (shared > before) flag_error(err, LORA_DEVERR_BAD_LEN);
    }
  }
  float q[kPer], acc[kPer];
  const bf16* qp = static_cast<const bf16*>(a.q) + t * a.q_stride + h * D + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = __bfloat162float(qp[i]) * a.scale;
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int lo = a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
  for (int j = lo > 0 && a.n_sink > 0 ? 0 : lo; j <= p; ++j) {
    if (j < lo && j >= a.n_sink) j = lo;
    const int row = j < shared ? shared_row : s;
    const int page = kv.block_table[static_cast<int64_t>(row) * kv.max_pages + j / kv.page_size];
    float dot = 0.f, v[kPer];
    const bool ok = page >= 0 && page < kv.n_pages;
    if (!ok) flag_error(err, LORA_DEVERR_BAD_PAGE);
    const int64_t at =
        ok ? ((static_cast<int64_t>(page) * kv.n_kv_heads + hk) * kv.page_size + j % kv.page_size) * D +
                 lane * kPer
           : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      dot += ok ? q[i] * __bfloat162float(static_cast<const bf16*>(kv.k_cache)[at + i]) : 0.f;
      v[i] = ok ? __bfloat162float(static_cast<const bf16*>(kv.v_cache)[at + i]) : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float m2 = fmaxf(m, dot), c = expf(m - m2), e = expf(dot - m2);
    l = l * c + e;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = acc[i] * c + e * v[i];
    m = m2;
  }
  bf16* o = static_cast<bf16*>(a.out) + t * a.out_stride + h * D + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = __float2bfloat16(l > 0.f ? acc[i] / l : 0.f);
}

}  // namespace

size_t attn_ws_bytes(const lora_paged_kv_t&, int, int) { return 16; }

cudaError_t launch_attn(const lora_paged_kv_t& kv, const AttnArgs& a, cudaStream_t st,
                        const DeviceInfo&) {
  const int64_t warps = static_cast<int64_t>(kv.T) * a.n_q_heads;
  const dim3 grid(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  uint32_t* err = static_cast<uint32_t*>(a.ws);
  if (kv.head_dim == 64)
    attn_kernel<64><<<grid, kWarps * 32, 0, st>>>(kv, a, err);
  else
    attn_kernel<128><<<grid, kWarps * 32, 0, st>>>(kv, a, err);
  return cudaGetLastError();
}

}  // namespace lora
