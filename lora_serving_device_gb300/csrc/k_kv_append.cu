// Rotation of q and k by position and the append of k and v to the paged
// cache, in one pass over the new tokens (lora_kv_append):
//   (a, b) -> (a c - b s, b c + a s) for pair i, c and s from the caller's
//   table at the position of the pair's axis; v is copied.
//
// Bound by memory: every value is read once and written once.  One block of
// 128 threads takes one token.  A thread owns one 16-value unit of a head
// (the two 8-value vectors that hold eight whole pairs: apart by rot_dim / 2
// in the half form, neighbours in the interleaved form and past rot_dim) and
// walks the heads with it, so the table's 16 values are loaded once for all
// its heads and every access is 16 bytes wide.  The loads of kBatch heads are
// in flight first; the lookups of the sequence, position and page, which they
// do not need, run beside them.
// Measured: a prompt of 8192, 32 / 8 heads of 128: 33.3 us, 6.2 TB/s of 6.69;
// 5238 tokens with 28 / 4 heads and three axes: 21.4 us, 4.6 TB/s (two heads a
// batch, for registers: four 23.0 us); 64 tokens 3.5 us.
#include "attn.cuh"

namespace lora {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 2;

struct Rot {
  float c[8], s[8];
};

template <bool kInter>
__device__ __forceinline__ void rotate(uint4& lo, uint4& hi, const Rot& r) {
  float a[8], b[8], x[8], y[8];
  load8(reinterpret_cast<const bf16*>(&lo), a);
  load8(reinterpret_cast<const bf16*>(&hi), b);
  if (kInter) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = a[2 * j] * r.c[j] - a[2 * j + 1] * r.s[j];
      x[2 * j + 1] = a[2 * j + 1] * r.c[j] + a[2 * j] * r.s[j];
      y[2 * j] = b[2 * j] * r.c[4 + j] - b[2 * j + 1] * r.s[4 + j];
      y[2 * j + 1] = b[2 * j + 1] * r.c[4 + j] + b[2 * j] * r.s[4 + j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = a[j] * r.c[j] - b[j] * r.s[j];
      y[j] = b[j] * r.c[j] + a[j] * r.s[j];
    }
  }
  lo = pack8_bf16(x);
  hi = pack8_bf16(y);
}

template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const lora_paged_kv_t kv,
                                                             const AppendArgs a) {
  constexpr int kUnits = D / 16;           // units of a head
  constexpr int kLanes = kThreads / kUnits;  // heads taken at once
  const int t = blockIdx.x;
  const int u = threadIdx.x % kUnits, h0 = threadIdx.x / kUnits;
  const bool rotates = 16 * u < a.rot_dim;
  const int o_lo = rotates && !kInter ? 8 * u : 16 * u;
  const int o_hi = rotates && !kInter ? a.rot_dim / 2 + 8 * u : 16 * u + 8;
  const int hq = a.n_q_heads, hk = kv.n_kv_heads, heads = hq + 2 * hk;

  pdl_wait();
  pdl_launch_dependents();

  const bf16* q = static_cast<const bf16*>(a.q) + t * a.q_stride;
  const bf16* k = static_cast<const bf16*>(a.k) + t * a.k_stride;
  const bf16* v = static_cast<const bf16*>(a.v) + t * a.v_stride;
  auto source = [&](int h) -> const bf16* {
    return h < hq ? q + h * D : h < hq + hk ? k + (h - hq) * D : v + (h - hq - hk) * D;
  };
  uint4 lo[kBatch], hi[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int hj = h + j * kLanes;
      if (hj < heads) {
        lo[j] = *reinterpret_cast<const uint4*>(source(hj) + o_lo);
        hi[j] = *reinterpret_cast<const uint4*>(source(hj) + o_hi);
      }
    }
  };
  load(h0);
  // (rows of no sequence are read, not used)
  const int s = seq_of_row(kv.q_off, kv.n_seqs, t);
  if (s < 0) return;
  const int p = kv.kv_len[s] - kv.q_off[s + 1] + t;
  Rot r;
  if (rotates) {
    auto pos_of = [&](int axis) {
      const int x = a.pos != nullptr ? a.pos[static_cast<int64_t>(axis) * kv.T + t] : p;
      if (x >= 0 && x < a.n_pos) return x;
      flag_error(a.err, LORA_DEVERR_BAD_POS);
      return -1;
    };
    auto axis_of = [&](int pair) {
      int ax = 0;
#pragma unroll
      for (int i = 0; i < LORA_MAX_POS_AXES - 1; ++i) ax += pair >= a.axis_end[i] ? 1 : 0;
      return ax < a.n_axes ? ax : a.n_axes - 1;
    };
    const int ax = axis_of(8 * u);
    if (ax == axis_of(8 * u + 7)) {
      const int x = pos_of(ax);
      if (x >= 0) {
        const float* row = a.cos_sin + static_cast<int64_t>(x) * a.rot_dim + 8 * u;
        load8(row, r.c);
        load8(row + a.rot_dim / 2, r.s);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.c[j] = 1.f, r.s[j] = 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int x = pos_of(axis_of(8 * u + j));
        const float* row = a.cos_sin + static_cast<int64_t>(x < 0 ? 0 : x) * a.rot_dim + 8 * u + j;
        r.c[j] = x < 0 ? 1.f : row[0];
        r.s[j] = x < 0 ? 0.f : row[a.rot_dim / 2];
      }
    }
  }

  // the row's place in the cache: element offset of its head 0, or -1
  int64_t place = -1;
  if (p >= 0) {
    const int col = p / kv.page_size;
    const int page = col < kv.max_pages
                         ? kv.block_table[static_cast<int64_t>(s) * kv.max_pages + col]
                         : -1;
    if (page >= 0 && page < kv.n_pages)
      place = (static_cast<int64_t>(page) * hk * kv.page_size + p % kv.page_size) * D;
    else
      flag_error(a.err, LORA_DEVERR_BAD_PAGE);
  }
  bf16* qo = static_cast<bf16*>(a.q_out) + t * a.q_out_stride;
  const int64_t head_step = static_cast<int64_t>(kv.page_size) * D;

  for (int h = h0; h < heads; h += kBatch * kLanes) {
    if (h != h0) load(h);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int hj = h + j * kLanes;
      if (hj >= heads) break;
      bf16* to;
      if (hj < hq) {
        to = qo + hj * D;
      } else {
        if (place < 0) continue;
        to = hj < hq + hk ? static_cast<bf16*>(kv.k_cache) + place + (hj - hq) * head_step
                          : static_cast<bf16*>(kv.v_cache) + place + (hj - hq - hk) * head_step;
      }
      if (rotates && hj < hq + hk) rotate<kInter>(lo[j], hi[j], r);
      *reinterpret_cast<uint4*>(to + o_lo) = lo[j];
      *reinterpret_cast<uint4*>(to + o_hi) = hi[j];
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const lora_paged_kv_t& kv, const AppendArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kv.T);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (kv.head_dim == 64)
    return a.interleaved ? cudaLaunchKernelEx(&cfg, kv_append_kernel<64, true>, kv, a)
                         : cudaLaunchKernelEx(&cfg, kv_append_kernel<64, false>, kv, a);
  return a.interleaved ? cudaLaunchKernelEx(&cfg, kv_append_kernel<128, true>, kv, a)
                       : cudaLaunchKernelEx(&cfg, kv_append_kernel<128, false>, kv, a);
}

}  // namespace lora
