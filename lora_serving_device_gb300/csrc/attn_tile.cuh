// Parts that the attention kernels' warps share: bounded waits, the TMA
// producer, values that no row sees, and writing, splitting and joining
// results.
#pragma once

#include "attn.cuh"
#include "ptx.cuh"

namespace lora {

constexpr uint64_t kAttnWaitNs = 2000000000ull;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ void named_bar(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// Whether any of the n threads at the barrier says so.
__device__ __forceinline__ bool named_any(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}
// Every lane waits (and so sees what the barrier orders); the same answer in
// all of them.  Once a wait of the CTA gave up the others return at once.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const bool ok = ptx::mbar_test_wait(bar, parity) ||
                  (!*abort && ptx::mbar_wait_bounded(bar, parity, abort, kAttnWaitNs));
  return __all_sync(0xffffffffu, ok);
}
// Bounds a polling loop in time: out() after each fruitless round.
struct Patience {
  uint32_t n = 0;
  uint64_t t0 = 0;
  __device__ __forceinline__ void reset() { n = 0; }
  __device__ __forceinline__ bool out(volatile int* abort) {
    if (++n < 4096u) return false;
    if (n == 4096u) t0 = ptx::globaltimer_ns();
    int stop = 0;
    if ((n & 255u) == 0u) {
      stop = *abort || ptx::globaltimer_ns() - t0 > kAttnWaitNs ? 1 : 0;
      if (stop) *abort = 1;
    }
    return __any_sync(0xffffffffu, stop);
  }
};

__device__ __forceinline__ bool tile_key_seen(const RowTile& t, int key) {
  return (key >= t.vis_lo && key <= t.vis_hi) || key < t.n_sink;
}

// The values of keys that no row of the tile sees are made zero in shared
// memory (their weights are zero, but 0 * NaN is not); what was not loaded
// too.  One warp, all lanes; V as the tensor map lays it out.
template <int D>
__device__ __forceinline__ void zero_unseen_values(const RowTile& t, int tile, uint8_t* V) {
  const int key0 = tile * kKeys;
  if (key0 >= t.vis_lo && key0 + kKeys - 1 <= t.vis_hi) return;
  __syncwarp();
  const int lane = threadIdx.x & 31;
  for (int r = lane; r < kKeys; r += 32) {
    if (tile_key_seen(t, key0 + r)) continue;
    uint8_t* row = V + (r / 8) * (D / 64) * 1024 + (r % 8) * 128;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int x = 0; x < 8; ++x)
        *reinterpret_cast<uint4*>(row + h * 1024 + x * 16) = make_uint4(0, 0, 0, 0);
  }
  ptx::fence_proxy_async_smem();
  __syncwarp();
}

// 4-D tiled load (c0 innermost), completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* tm, uint64_t* bar,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %3, %3, %4}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(tm), "r"(ptx::smem_u32(bar)), "r"(0), "r"(c3)
      : "memory");
}

// c1 is the head, c2 the token, c3 the 64-value half of the head.
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* tm, uint64_t* bar,
                                              int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(tm), "r"(ptx::smem_u32(bar)), "r"(0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Brings in the K or V rows of a key tile: a box per page (or per 128 rows of a
// larger one), each box in the hands of a lane, which looks its page up.
// Pages that no row sees are not touched.  A page that is missing is asked for
// past the cache's end, where the tensor map reads zeros.  One warp.
template <int D>
struct TileLoader {
  int page, lg_page, box, boxes;
  __device__ __forceinline__ explicit TileLoader(const AttnParams& P)
      : page(P.kv.page_size),
        lg_page(P.lg_page),
        box(page < kKeys ? page : kKeys),
        boxes(kKeys / box) {}
  // Where this lane's box of the segment's i-th tile starts in the cache, in
  // groups of eight rows; -1: not needed.
  __device__ __forceinline__ int lookup(const AttnParams& P, const Segment& g, int i) const {
    const int lane = threadIdx.x & 31;
    const int key0 = key_tile(g.t, g.first + i) * kKeys + lane * box;
    if (lane >= boxes || !((key0 <= g.t.vis_hi && key0 + box - 1 >= g.t.vis_lo) ||
                           key0 < g.t.n_sink))
      return -1;
    const int id =
        P.kv.block_table[static_cast<int64_t>(g.table_row) * P.kv.max_pages + (key0 >> lg_page)];
    if (id < 0 || id >= P.kv.n_pages) {
      flag_error(P.err, LORA_DEVERR_BAD_PAGE);
      return P.kv.n_pages * P.kv.n_kv_heads * (page / 8);
    }
    return (id * P.kv.n_kv_heads + g.head) * (page / 8) + (key0 & (page - 1)) / 8;
  }
  __device__ __forceinline__ void load(const CUtensorMap* tm, uint64_t* full, uint8_t* dst,
                                       int at) const {
    const int lane = threadIdx.x & 31;
    const uint32_t bytes = static_cast<uint32_t>(box) * D * 2;
    const uint32_t all = __popc(__ballot_sync(0xffffffffu, at >= 0)) * bytes;
    if (lane == 0) ptx::mbar_arrive_expect_tx(full, all);
    __syncwarp();
    if (at >= 0) tma_load_4d(dst + lane * bytes, tm, full, at);
  }
};

// Value d of row n of a finished item: o / sum.  The prefix phase keeps it in
// fp32 with its log-sum-exp (log2 units, m + log2 sum); otherwise it is joined
// with that part, if there is one, and rounded to out.
template <int D>
__device__ __forceinline__ void write_row(const AttnParams& P, const Segment& g, int n, int d,
                                          float o, float sum, float m) {
  const int r = g.t.row0 + n;
  const int64_t t = g.tok0 + r / P.group;
  const int h = g.head * P.group + r % P.group;
  float x = sum > 0.f ? o / sum : 0.f;
  if (P.groups_phase || g.shared) {
    const float lse = sum > 0.f ? m + log2f(sum) : -INFINITY;
    const int64_t at = t * P.n_q_heads + h;
    if (P.groups_phase) {
      P.prior[at * D + d] = x;
      if (d == 0) P.prior_lse[at] = lse;
      return;
    }
    const float other = P.prior_lse[at], top = fmaxf(lse, other);
    if (top > -INFINITY) {
      const float a = exp2f(lse - top), b = exp2f(other - top);
      x = (a * x + b * P.prior[at * D + d]) / (a + b);
    }
  }
  P.out[t * P.out_stride + h * D + d] = __float2bfloat16_rn(x);
}

// The same for a thread that holds a whole row, eight values at a time.
template <int D>
struct RowWriter {
  float own, other;  // factors of this result and of the prior part
  bf16* out;
  float* prior;
  bool to_prior, join;
  __device__ __forceinline__ RowWriter(const AttnParams& P, const Segment& g, int n, float m,
                                       float sum) {
    const int r = g.t.row0 + n;
    const int64_t t = g.tok0 + r / P.group;
    const int h = g.head * P.group + r % P.group;
    to_prior = P.groups_phase;
    join = !to_prior && g.shared;
    own = sum > 0.f ? 1.f / sum : 0.f;
    other = 0.f;
    out = P.out + t * P.out_stride + h * D;
    const int64_t at = t * P.n_q_heads + h;
    prior = P.prior + at * D;
    if ((to_prior || join) && n < g.t.n_rows) {
      const float lse = sum > 0.f ? m + log2f(sum) : -INFINITY;
      if (to_prior) {
        P.prior_lse[at] = lse;
      } else {
        const float lp = P.prior_lse[at], top = fmaxf(lse, lp);
        if (top > -INFINITY) {
          const float a = exp2f(lse - top), b = exp2f(lp - top);
          own *= a / (a + b);
          other = b / (a + b);
        }
      }
    }
  }
  __device__ __forceinline__ void write8(int d, const float* x) const {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * own;
    if (to_prior) {
      store8(prior + d, y);
      return;
    }
    if (join) {
      float z[8];
      load8(prior + d, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += other * z[i];
    }
    store8(out + d, y);
  }
};

// The slot of the item's c-th part.
__device__ __forceinline__ int64_t part_slot(const Segment& g, int c) {
  return static_cast<int64_t>(g.cta0 + c) * 2 + (c == 0 ? 1 : 0);
}

// Threads of named barrier `bar` (cnt of them) have written this CTA's part:
// is it the last of the item (or of its half)?  Leaves the counter at zero.
__device__ __forceinline__ bool last_to_arrive(const AttnParams& P, const Segment& g, int counter,
                                               bool leader, int* flag, int bar, int cnt) {
  __threadfence();
  named_bar(bar, cnt);
  if (leader) {
    const uint32_t before = atomicAdd(&P.count[counter], 1u);
    *flag = before + 1 == static_cast<uint32_t>(g.parts) ? 1 : 0;
    if (*flag) P.count[counter] = 0;
    __threadfence();
  }
  named_bar(bar, cnt);
  __threadfence();
  return *flag != 0;
}

// Maximum and sum of row n over the item's parts.
template <int kRows>
__device__ __forceinline__ void merged_max(const AttnParams& P, const Segment& g, int n, float* m,
                                           float* sum) {
  float top = -INFINITY, s = 0.f;
  for (int c = 0; c < g.parts; ++c)
    top = fmaxf(top, __ldcg(P.part_ml + (part_slot(g, c) * kRows + n) * 2));
  if (top > -INFINITY) {
    for (int c = 0; c < g.parts; ++c) {
      const float2 ml =
          __ldcg(reinterpret_cast<const float2*>(P.part_ml + (part_slot(g, c) * kRows + n) * 2));
      s += exp2f(ml.x - top) * ml.y;
    }
  }
  *m = top;
  *sum = s;
}

// Value d of row n summed over the item's parts, in their order.
template <int kRows, int D>
__device__ __forceinline__ float merged_value(const AttnParams& P, const Segment& g, int n, int d,
                                              float top) {
  float o = 0.f;
  if (top == -INFINITY) return o;
#pragma unroll 4
  for (int c = 0; c < g.parts; ++c) {
    const int64_t row = part_slot(g, c) * kRows + n;
    const float f = exp2f(__ldcg(P.part_ml + row * 2) - top);
    // a part that saw nothing of this row holds 0 at most
    o += f * __ldcg(P.part + row * D + d);
  }
  return o;
}

}  // namespace lora
