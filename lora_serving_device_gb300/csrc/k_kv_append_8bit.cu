// Rotation of q and k by position and the append of k and v to the 8-bit paged
// cache, in one pass over the new tokens (lora_kv_append_8bit).
//
// A scale block is kScaleBlock tokens of a head; a run is the rows of the call that
// fall into one.  For a run and a head:
//   byte = max(scale_byte(max |x|), the block's byte if it holds earlier rows)
//   code = e4m3(x 2^(127 - byte)),  x the rotated fp32 value (k) or v
// and the codes of earlier rows are moved to the scale if it grew.
//
// A warp takes a run and a head: its rows stay in registers, as they come, between the maximum
// and the codes, and the maximum is one reduction over the warp (a key is rotated twice for it:
// that costs less than the registers that would keep it).  Lanes split a row into 16-value
// units (two vectors of eight that hold whole pairs), 32 / units rows at once.  q's rows go
// by in the same blocks, by the same units.  A block of warps takes kRows rows of the batch, 16
// where there are prompts and else one, and a share of their heads (gridDim.y); the
// rows' cosines and sines wait in shared memory.
//
// Bound by memory: every value is read once and written once, k and v in half the bytes.
// Measured: prompt of 8192, 32 / 8 heads of 128: 39 us, 4.8 TB/s of 6.69 (lookups, then loads
// that the few warps which 128 registers leave room for do not keep in flight all the time; more
// warps with fewer registers took longer, 48 us at 96); 5238 tokens of 28 / 4 heads, three
// axes: 23.4 us, 3.5 TB/s; 64 tokens 4.9 us.
#include <algorithm>

#include "attn.cuh"
#include "fp8.cuh"
#include "rotary.cuh"

namespace lora {
namespace {

constexpr int kWarps = 4, kBlocksPerSm = 4;
constexpr int kMaxRot = 128;

struct RunInfo {
  int64_t page;   // of the row in the cache; -1: missing, or not cached
  int in_seq;     // 0: the row belongs to no sequence
  int p;          // position
  int run;        // rows of the run that begins here; 0: none does
};

// Row t of the batch, by one thread.
__device__ __forceinline__ RunInfo row_info(const lora_paged_kv_t& kv, int t, int s, int block,
                                            uint32_t* err) {
  RunInfo x = {-1, 1, 0, 0};
  const int begin = kv.q_off[s], end = kv.q_off[s + 1];
  if (end <= t) {  // offsets out of order: s is not the row's sequence, and a run would have no rows
    flag_error(err, LORA_DEVERR_BAD_LEN);
    x.in_seq = 0;
    return x;
  }
  x.p = kv.kv_len[s] - end + t;
  if (x.p < 0) return x;
  const int col = x.p / kv.page_size;
  const int page =
      col < kv.max_pages ? kv.block_table[static_cast<int64_t>(s) * kv.max_pages + col] : -1;
  if (page >= 0 && page < kv.n_pages)
    x.page = page;
  else
    flag_error(err, LORA_DEVERR_BAD_PAGE);
  if (t == begin || x.p % block == 0) x.run = min(min(end, kv.T) - t, block - x.p % block);
  return x;
}

// The cosines and sines of a row at position p, by one warp: rot_dim of them, as in the table.
__device__ __forceinline__ void stage_rot(const AppendArgs& a, int T, int t, int p, float* to) {
  const int half = a.rot_dim / 2;
  for (int i = threadIdx.x & 31; i < half; i += 32) {
    int axis = 0;
#pragma unroll
    for (int n = 0; n < LORA_MAX_POS_AXES - 1; ++n) axis += i >= a.axis_end[n] ? 1 : 0;
    axis = min(axis, a.n_axes - 1);
    const int x = a.pos != nullptr ? a.pos[static_cast<int64_t>(axis) * T + t] : p;
    const bool ok = x >= 0 && x < a.n_pos;
    if (!ok) flag_error(a.err, LORA_DEVERR_BAD_POS);
    const float* row = a.cos_sin + static_cast<int64_t>(ok ? x : 0) * a.rot_dim + i;
    to[i] = ok ? row[0] : 1.f;
    to[half + i] = ok ? row[half] : 0.f;
  }
}

// A unit as it was loaded, rotated with its eight pairs' cosines and sines if there are any.
template <bool kInter>
__device__ __forceinline__ void unit_values(const uint4 (&raw)[2], const float* cos,
                                            const float* sin, float (&x)[16]) {
  load8(reinterpret_cast<const bf16*>(&raw[0]), *reinterpret_cast<float(*)[8]>(x));
  load8(reinterpret_cast<const bf16*>(&raw[1]), *reinterpret_cast<float(*)[8]>(x + 8));
  if (cos == nullptr) return;
  Rot r;
  load8(cos, r.c);
  load8(sin, r.s);
  rotate_unit<kInter>(x, r);
}

template <int D, bool kInter, int kRows>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm) kv_append_8bit_kernel(const lora_paged_kv_t kv,
                                                                        const AppendArgs a) {
  constexpr int kUnits = D / 16;          // of a row
  constexpr int kAtOnce = 32 / kUnits;    // rows, or heads, that a warp takes at once
  constexpr int kTrips = kScaleBlock / kAtOnce;
  constexpr int kStaged = kRows + kScaleBlock - 1;  // (the last run may go on behind the rows)
  __shared__ RunInfo info[kRows];
  __shared__ alignas(16) float table[kStaged][kMaxRot];
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

  // q: lanes take rows of a head where there are rows enough, heads of a row else.  The
  // first heads' loads begin here, beside the lookups that follow.
  constexpr bool kByRow = kRows >= kAtOnce;
  constexpr int kGroups = kByRow ? kRows / kAtOnce : 1;  // of rows
  constexpr int kAhead = kByRow ? 4 : 2;                 // heads whose loads are in flight
  static_assert(kWarps % kGroups == 0, "");
  const int q_row = kByRow ? (warp % kGroups) * kAtOnce + r0 : 0;
  const int n_warps = gridDim.y * kWarps / kGroups;  // that share a group's heads
  const int q_warp = (blockIdx.y * kWarps + warp) / kGroups;
  const int q_first = kByRow ? q_warp : q_warp * kAtOnce + r0;
  const int q_step = kByRow ? n_warps : n_warps * kAtOnce;
  const bf16* q_from = static_cast<const bf16*>(a.q) + static_cast<int64_t>(t0 + q_row) * a.q_stride;
  uint4 q_raw[kAhead][2];
  auto load_q = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h0 + k * q_step < hq) {
        q_raw[k][0] = *reinterpret_cast<const uint4*>(q_from + (h0 + k * q_step) * D + o_lo);
        q_raw[k][1] = *reinterpret_cast<const uint4*>(q_from + (h0 + k * q_step) * D + o_hi);
      }
  };
  if (t0 + q_row < kv.T) load_q(q_first);  // (rows of no sequence are read, not used)

  if (warp == 0) {
    if constexpr (kRows == 1) {
      const int s = seq_of_row(kv.q_off, kv.n_seqs, t0);
      if (lane == 0) info[0] = s >= 0 ? row_info(kv, t0, s, block, a.err) : RunInfo{-1, 0, 0, 0};
    } else if (lane < kRows) {
      const int t = t0 + lane;
      RunInfo x = {-1, 0, 0, 0};
      if (t < kv.T && t >= kv.q_off[0] && t < kv.q_off[kv.n_seqs]) {
        int lo = 0, hi = kv.n_seqs;  // q_off[lo] <= t < q_off[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (kv.q_off[mid] <= t) lo = mid; else hi = mid;
        }
        x = row_info(kv, t, lo, block, a.err);
      }
      info[lane] = x;
    }
  }
  __syncthreads();
  if (a.rot_dim > 0) {
    for (int i = warp; i < kStaged; i += kWarps) {
      // rows behind the block's: of a run that began in it
      int p = -1;
      bool wanted = false;
      if (i < kRows) {
        wanted = info[i].in_seq != 0;
        p = info[i].p;
      } else {
        for (int j = 0; j < kRows; ++j)
          if (j + info[j].run > i) {
            wanted = true;
            p = info[j].p + i - j;
          }
      }
      if (wanted) stage_rot(a, kv.T, t0 + i, p, table[i]);
    }
    __syncthreads();
  }
  auto cos_of = [&](int row) { return rotates ? &table[row][8 * u] : nullptr; };
  auto sin_of = [&](int row) { return &table[row][a.rot_dim / 2 + 8 * u]; };

  if (hq > 0 && info[q_row].in_seq) {
    bf16* to = static_cast<bf16*>(a.q_out) + static_cast<int64_t>(t0 + q_row) * a.q_out_stride;
    for (int h0 = q_first; h0 < hq; h0 += kAhead * q_step) {
      uint4 raw[kAhead][2];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) raw[k][0] = q_raw[k][0], raw[k][1] = q_raw[k][1];
      load_q(h0 + kAhead * q_step);
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (h0 + k * q_step < hq) {
          float x[16];
          unit_values<kInter>(raw[k], cos_of(q_row), sin_of(q_row), x);
          store8(to + (h0 + k * q_step) * D + o_lo, x);
          store8(to + (h0 + k * q_step) * D + o_hi, x + 8);
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
      const int64_t stride = is_k ? a.k_stride : a.v_stride;
      const bf16* from = static_cast<const bf16*>(is_k ? a.k : a.v) + (t0 + i) * stride + h * D;
      const int64_t head = me.page * hk + h;
      const int first = me.p % kv.page_size;  // the run's first row in the page
      uint8_t* cache = static_cast<uint8_t*>(is_k ? kv.k_cache : kv.v_cache) +
                       (head * kv.page_size + first) * D;
      uint8_t* scale = (is_k ? a.k_scale : a.v_scale) + head * (kv.page_size / block) + first / block;
      const int held = first % block;  // earlier rows of the block
      uint4 raw[kTrips][2];
#pragma unroll
      for (int k = 0; k < kTrips; ++k) {
        const int row = k * kAtOnce + r0;
        raw[k][0] = raw[k][1] = make_uint4(0, 0, 0, 0);
        if (row < me.run) {
          raw[k][0] = *reinterpret_cast<const uint4*>(from + row * stride + o_lo);
          raw[k][1] = *reinterpret_cast<const uint4*>(from + row * stride + o_hi);
        }
      }
      const int old = held > 0 ? scale_read(*scale) : 0;
      auto values = [&](int k, float (&x)[16]) {
        const int row = min(k * kAtOnce + r0, me.run - 1);
        unit_values<kInter>(raw[k], is_k ? cos_of(i + row) : nullptr, sin_of(i + row), x);
      };
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < kTrips; ++k) {
        float x[16];
        values(k, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(x[j]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fminf(top, 3.4028235e38f);
      const int byte = max(scale_byte(top), old);
      const float inv = scale_of(254 - byte);
#pragma unroll
      for (int k = 0; k < kTrips; ++k) {
        const int row = k * kAtOnce + r0;
        if (row >= me.run) continue;
        float x[16];
        values(k, x);
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          c[j] = pack4_e4m3(x[4 * j] * inv, x[4 * j + 1] * inv, x[4 * j + 2] * inv,
                            x[4 * j + 3] * inv);
        *reinterpret_cast<uint2*>(cache + row * D + o_lo) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2*>(cache + row * D + o_hi) = make_uint2(c[2], c[3]);
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
  // Heads are shared out as far as all blocks of warps stay resident at once: the lookups at
  // their beginning take longer than the rest of a small one (prompt of 8192, 512 blocks: 39
  // us, shared by two 46, by four 56; 5238 tokens of 28 + 2 x 4 heads: 29, by two 23).
  const int blocks = (kv.T + kScaleBlock - 1) / kScaleBlock;
  const int share = (kDecodeScheduleCtas * kBlocksPerSm + blocks / 2) / blocks;
  cfg.gridDim = prompts ? dim3(blocks, std::min(4, std::max(1, share))) : dim3(kv.T, 4);
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
