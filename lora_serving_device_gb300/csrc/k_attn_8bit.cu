// Attention over the paged cache in 8 bits (lora_attn_paged_8bit,
// lora_attn_prefix_8bit), the plain kernel: a block to a row and query head, a
// thread to a key, then a thread to a value of the result.
//   s_j = c q . code_j 2^(kb_j - 127),  out = sum_j p_j 2^(vb_j - 127) code_j / sum_j p_j
// with the running maximum and sum of a softmax in one pass, in 32 bits.
#include "attn.cuh"
#include "fp8.cuh"

namespace lora {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) attn_8bit_kernel(const lora_paged_kv_t kv,
                                                             const AttnArgs a) {
  __shared__ float q[D], p[kThreads], vs[kThreads], red[kThreads / 32];
  __shared__ int64_t rows[kThreads];
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  uint32_t* err = static_cast<uint32_t*>(a.ws);
  const int s = seq_of_row(kv.q_off, kv.n_seqs, t);
  if (s < 0) return;
  const int hk = kv.n_kv_heads, kh = h / (a.n_q_heads / hk);
  const int block = kv.page_size < kScaleBlock ? kv.page_size : kScaleBlock;
  const int64_t cap = static_cast<int64_t>(kv.max_pages) * kv.page_size;
  int len = kv.kv_len[s];
  if (len > cap) {
    if (tid == 0) flag_error(err, LORA_DEVERR_BAD_LEN);
    len = static_cast<int>(cap);
  }
  const int pos = min(len - (kv.q_off[s + 1] - t), len - 1);
  int shared = 0, first_seq = s;
  for (int g = 0; g < a.n_groups; ++g)
    if (a.group_off[g] <= s && s < a.group_off[g + 1]) {
      first_seq = a.group_off[g];
      shared = a.prefix_len[g];
    }
  if (shared > len - (kv.q_off[s + 1] - kv.q_off[s]) && shared > 0 && tid == 0) flag_error(err, LORA_DEVERR_BAD_LEN);
  if (tid < D) q[tid] = __bfloat162float(static_cast<const bf16*>(a.q)[t * a.q_stride + h * D + tid]) * a.scale;
  const int lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
  float m = -INFINITY, l = 0.f, o = 0.f;
  __syncthreads();
  for (int j0 = 0; j0 <= pos; j0 += kThreads) {
    const int j = j0 + tid;
    const bool seen = j <= pos && (j >= lo || j < a.n_sink);
    if (j0 + kThreads <= lo && j0 >= a.n_sink) continue;
    float x = -INFINITY;
    int64_t row = -1;
    if (seen) {
      const int64_t entry = (j < shared ? first_seq : s) * static_cast<int64_t>(kv.max_pages) + j / kv.page_size;
      const int page = kv.block_table[entry];
      x = 0.f;
      if (page >= 0 && page < kv.n_pages) {
        const int64_t head = static_cast<int64_t>(page) * hk + kh;
        const int in = j % kv.page_size;
        row = (head * kv.page_size + in) * D;
        const int64_t at = head * (kv.page_size / block) + in / block;
        const uint32_t* k = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(kv.k_cache) + row);
        for (int i = 0; i < D / 4; ++i) {
          const float2 u = unpack2_e4m3(k[i]), v = unpack2_e4m3(k[i] >> 16);
          x += q[4 * i] * u.x + q[4 * i + 1] * u.y + q[4 * i + 2] * v.x + q[4 * i + 3] * v.y;
        }
        x *= scale_of(scale_read(a.k_scale[at]));
        vs[tid] = scale_of(scale_read(a.v_scale[at]));
      } else {
        flag_error(err, LORA_DEVERR_BAD_PAGE);
      }
    }
    rows[tid] = row;
    float mx = x;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
    if ((tid & 31) == 0) red[tid / 32] = mx;
    __syncthreads();
    const float now = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float f = m == -INFINITY ? 0.f : __expf(m - now);
    p[tid] = seen ? __expf(x - now) : 0.f;
    m = now;
    __syncthreads();
    l *= f;
    o *= f;
    for (int i = 0; i < kThreads; ++i) {
      l += p[i];
      if (tid < D && p[i] > 0.f && rows[i] >= 0) {
        const uint8_t c = static_cast<const uint8_t*>(kv.v_cache)[rows[i] + tid];
        o += p[i] * vs[i] * unpack2_e4m3(c).x;
      }
    }
    __syncthreads();
  }
  if (tid < D)
    static_cast<bf16*>(a.out)[t * a.out_stride + h * D + tid] = __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
}

}  // namespace

cudaError_t launch_attn_8bit(const lora_paged_kv_t& kv, const AttnArgs& a, cudaStream_t st) {
  const dim3 grid(kv.T, a.n_q_heads);
  if (kv.head_dim == 64)
    attn_8bit_kernel<64><<<grid, kThreads, 0, st>>>(kv, a);
  else
    attn_8bit_kernel<128><<<grid, kThreads, 0, st>>>(kv, a);
  return cudaGetLastError();
}

}  // namespace lora
