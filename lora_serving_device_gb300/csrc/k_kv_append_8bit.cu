// Rotation of q and k by position and the append of k and v to the 8-bit paged
// cache, in one pass over the new tokens (lora_kv_append_8bit).
//
// A scale block is kScaleBlock tokens of a head; a run is the rows of the call that
// fall into one.  For a run and a head:
//   byte = max(scale_byte(max |x|), the block's byte if it holds earlier rows)
//   code = e4m3(x 2^(127 - byte)),  x the rotated fp32 value (k) or v
// and the codes of earlier rows are moved to the scale if it grew.
//
// A warp takes a run and a head: its rows stay in registers between the maximum and
// the codes, and the maximum is one reduction over the warp.  Lanes split a row into
// 16-value units (two vectors of eight that hold whole pairs), 32 / units rows at once.
// q's rows go by in the same blocks, by the same units.  A block of warps takes kRows
// rows of the batch: 16 where there are prompts, else one.
//
// Bound by memory: every value is read once and written once, k and v in half the bytes.
#include "attn.cuh"
#include "fp8.cuh"
#include "rotary.cuh"

namespace lora {
namespace {

constexpr int kWarps = 4;

struct RunInfo {
  int64_t page;   // of the row in the cache; -1: missing, or not cached
  int seq_rows;   // 0: the row belongs to no sequence
  int p;          // position
  int run;        // rows of the run that begins here; 0: none does
};

template <int D, bool kInter, int kRows>
__global__ void __launch_bounds__(kWarps * 32) kv_append_8bit_kernel(const lora_paged_kv_t kv,
                                                                     const AppendArgs a) {
  constexpr int kUnits = D / 16;          // of a row
  constexpr int kAtOnce = 32 / kUnits;    // rows, or heads, that a warp takes at once
  constexpr int kTrips = kScaleBlock / kAtOnce;
  __shared__ RunInfo info[kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int u = lane % kUnits, r0 = lane / kUnits;
  const int t0 = blockIdx.x * kRows;
  const bool rotates = 16 * u < a.rot_dim;
  const int o_lo = rotates && !kInter ? 8 * u : 16 * u;
  const int o_hi = rotates && !kInter ? a.rot_dim / 2 + 8 * u : 16 * u + 8;
  const int block = kv.page_size < kScaleBlock ? kv.page_size : kScaleBlock;
  const int hq = a.n_q_heads, hk = kv.n_kv_heads;

  pdl_wait();
  pdl_launch_dependents();

  for (int i = warp; i < kRows; i += kWarps) {
    const int t = t0 + i;
    RunInfo x = {-1, 0, 0, 0};
    const int s = t < kv.T ? seq_of_row(kv.q_off, kv.n_seqs, t) : -1;
    if (s >= 0) {
      const int begin = kv.q_off[s], end = min(kv.q_off[s + 1], kv.T);
      x.seq_rows = 1;
      x.p = kv.kv_len[s] - kv.q_off[s + 1] + t;
      if (x.p >= 0) {
        const int col = x.p / kv.page_size;
        const int page = col < kv.max_pages
                             ? kv.block_table[static_cast<int64_t>(s) * kv.max_pages + col]
                             : -1;
        if (page >= 0 && page < kv.n_pages)
          x.page = page;
        else
          flag_error(a.err, LORA_DEVERR_BAD_PAGE);
        if (t == begin || x.p % block == 0) x.run = min(end - t, block - x.p % block);
      }
    }
    if (lane == 0) {
      info[i] = x;
      if (x.seq_rows && x.page < 0) flag_bad_pos(a, kv.T, t, x.p);
    }
  }
  __syncthreads();

  auto load = [&](const bf16* head, float (&x)[16]) {
    load8(head + o_lo, *reinterpret_cast<float(*)[8]>(x));
    load8(head + o_hi, *reinterpret_cast<float(*)[8]>(x + 8));
  };

  // ---- q: lanes take rows of a head where there are rows enough, heads of a row else
  if (hq > 0) {
    constexpr bool kByRow = kRows >= kAtOnce;
    constexpr int kGroups = kByRow ? kRows / kAtOnce : 1;  // of rows
    static_assert(kWarps % kGroups == 0, "");
    const int row = kByRow ? (warp % kGroups) * kAtOnce + r0 : 0;
    const int n_warps = gridDim.y * kWarps / kGroups;  // that share a group's heads
    const int w = (blockIdx.y * kWarps + warp) / kGroups;
    const int first = kByRow ? w : w * kAtOnce + r0, step = kByRow ? n_warps : n_warps * kAtOnce;
    const RunInfo me = info[row];
    if (me.seq_rows) {
      const int64_t t = t0 + row;
      Rot rot;
      if (rotates) load_rot(a, kv.T, t0 + row, me.p, u, rot);
      const bf16* from = static_cast<const bf16*>(a.q) + t * a.q_stride;
      bf16* to = static_cast<bf16*>(a.q_out) + t * a.q_out_stride;
#pragma unroll 2
      for (int h = first; h < hq; h += step) {
        float x[16];
        load(from + h * D, x);
        if (rotates) rotate_unit<kInter>(x, rot);
        store8(to + h * D + o_lo, x);
        store8(to + h * D + o_hi, x + 8);
      }
    }
  }

  // ---- k and v: a warp to a run and a head
  for (int i = 0; i < kRows; ++i) {
    const RunInfo me = info[i];
    if (me.run == 0 || me.page < 0) continue;
    for (int task = blockIdx.y * kWarps + warp; task < 2 * hk; task += gridDim.y * kWarps) {
      const bool is_k = task < hk;
      const int h = is_k ? task : task - hk;
      const bf16* from = static_cast<const bf16*>(is_k ? a.k : a.v) +
                         static_cast<int64_t>(t0 + i) * (is_k ? a.k_stride : a.v_stride) + h * D;
      const int64_t stride = is_k ? a.k_stride : a.v_stride;
      const int64_t head = me.page * hk + h;
      const int first = me.p % kv.page_size;  // the run's first row in the page
      uint8_t* cache = static_cast<uint8_t*>(is_k ? kv.k_cache : kv.v_cache) +
                       (head * kv.page_size + first) * D;
      uint8_t* scale = (is_k ? a.k_scale : a.v_scale) + head * (kv.page_size / block) + first / block;
      const int held = first % block;  // earlier rows of the block
      const int old = held > 0 ? scale_read(*scale) : 0;
      float x[kTrips][16];
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < kTrips; ++k) {
        const int row = k * kAtOnce + r0;
        if (row < me.run) {
          load(from + row * stride, x[k]);
          if (is_k && rotates) {
            Rot rot;
            load_rot(a, kv.T, t0 + i + row, me.p + row, u, rot);
            rotate_unit<kInter>(x[k], rot);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(x[k][j]));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fminf(top, 3.4028235e38f);
      const int byte = max(scale_byte(top), old);
      const float inv = scale_of(254 - byte);
#pragma unroll
      for (int k = 0; k < kTrips; ++k) {
        const int row = k * kAtOnce + r0;
        if (row < me.run) {
          uint32_t c[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            c[j] = pack4_e4m3(x[k][4 * j] * inv, x[k][4 * j + 1] * inv, x[k][4 * j + 2] * inv,
                              x[k][4 * j + 3] * inv);
          *reinterpret_cast<uint2*>(cache + row * D + o_lo) = make_uint2(c[0], c[1]);
          *reinterpret_cast<uint2*>(cache + row * D + o_hi) = make_uint2(c[2], c[3]);
        }
      }
      if (byte > old) {
        if (old > 0) {  // the earlier rows' codes, to the new scale
          const int down = 127 - (byte - old);
          const float f = down > 0 ? scale_of(down) : 0.f;
          for (int o = lane * 4; o < held * D; o += 128) {
            uint32_t* at = reinterpret_cast<uint32_t*>(cache - held * D + o);
            const float2 lo = unpack2_e4m3(*at), hi = unpack2_e4m3(*at >> 16);
            *at = pack4_e4m3(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
          }
        }
        if (lane == 0) *scale = static_cast<uint8_t>(byte);
      }
    }
  }
}

template <int D, bool kInter>
cudaError_t launch(const lora_paged_kv_t& kv, const AppendArgs& a, cudaStream_t st) {
  const bool prompts = kv.max_q_len >= kScaleBlock;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = prompts ? dim3((kv.T + kScaleBlock - 1) / kScaleBlock, 4) : dim3(kv.T, 2);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return prompts ? cudaLaunchKernelEx(&cfg, kv_append_8bit_kernel<D, kInter, kScaleBlock>, kv, a)
                 : cudaLaunchKernelEx(&cfg, kv_append_8bit_kernel<D, kInter, 1>, kv, a);
}

}  // namespace

cudaError_t launch_kv_append_8bit(const lora_paged_kv_t& kv, const AppendArgs& a, cudaStream_t st) {
  if (kv.head_dim == 64)
    return a.interleaved ? launch<64, true>(kv, a, st) : launch<64, false>(kv, a, st);
  return a.interleaved ? launch<128, true>(kv, a, st) : launch<128, false>(kv, a, st);
}

}  // namespace lora
