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
// Once a wait of the CTA gave up, the others return at once.  One loop of few
// instructions: the roles' loops run side by side, and what they take together
// has to fit the instruction caches (with the loop doubled, a quick one before
// one that minds the clock, prompts are slower by 3 to 10%).
__device__ __forceinline__ void wait_quiet(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint32_t n = 0, t0 = 0;
#pragma unroll 1
  while (!ptx::mbar_try_wait(bar, parity) && !*abort) {
    if ((++n & 4095u) != 0u) continue;
    const uint32_t now = static_cast<uint32_t>(ptx::globaltimer_ns() >> 10);
    if (n == 4096u) t0 = now;
    if (now - t0 > static_cast<uint32_t>(kAttnWaitNs >> 10)) *abort = 1;
  }
}
// Every lane waits (and so sees what the barrier orders); false, in all of
// them, once a wait of the CTA gave up.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort) {
  wait_quiet(bar, parity, abort);
  return __all_sync(0xffffffffu, *abort == 0);
}
// One lane of a converged warp, in a form the compiler knows to be one thread.
// A loop that runs wholly inside such a branch issues an MMA in ~20 cycles; in
// one that lane 0 runs, or that a warp runs with a branch around the MMAs, each
// takes ~55 (8 MMAs of 128 x 128 x 16 on an idle pipe: 175 against 435 to 470).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// Shared-memory matrix descriptors in halves: the low words hold the address
// and the leading offset, the high words the stride and the 128-byte swizzle.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | (((lbo_bytes >> 4) & 0x3FFFu) << 16);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo_bytes) {
  return ((sbo_bytes >> 4) & 0x3FFFu) | (1u << 14) | (2u << 29);
}
// D[tmem] (+)= A[smem] B[smem] and A[tmem] B[smem], descriptors in halves.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                       uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Bounds one thread's polling loop in time: out() after each fruitless round.
struct Patience {
  uint32_t n = 0;
  uint64_t t0 = 0;
  __device__ __forceinline__ void reset() { n = 0; }
  __device__ __forceinline__ bool out(volatile int* abort) {
    if (++n < 4096u) return false;
    if (n == 4096u) t0 = ptx::globaltimer_ns();
    if ((n & 255u) != 0u) return false;
    if (!*abort && ptx::globaltimer_ns() - t0 <= kAttnWaitNs) return false;
    *abort = 1;
    return true;
  }
};

// Whether some row sees the key at place v.
__device__ __forceinline__ bool place_seen(const RowTile& t, int v) {
  const int key = window_key(t, v);
  return (key >= t.vis_lo && key <= t.vis_hi) || v < t.n_sink;
}

// Whether a key tile holds keys that no row of the row tile sees.
__device__ __forceinline__ bool tile_has_unseen(const RowTile& t, int v0) {
  return window_key(t, v0) < t.vis_lo || window_key(t, v0 + kKeys - 1) > t.vis_hi;
}
// The values of key `j` of such a tile are made zero in shared memory if no row
// sees the key (its weights are zero, but 0 * NaN is not): rows of the cache
// past the length or before the window, and what was not loaded at all.  V as
// the tensor map lays it out; the caller fences before the MMA reads it.
template <int D>
__device__ __forceinline__ void zero_unseen_value(const RowTile& t, int v0, int j, uint8_t* V) {
  if (place_seen(t, v0 + j)) return;
  uint8_t* row = V + (j / 8) * (D / 64) * 1024 + (j % 8) * 128;
  // (each lane starts elsewhere in its 128 bytes: the rows lie 128 bytes apart)
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
#pragma unroll
    for (int x = 0; x < 8; ++x)
      *reinterpret_cast<uint4*>(row + h * 1024 + ((x + j) & 7) * 16) = make_uint4(0, 0, 0, 0);
}

// L2 policies: what one CTA alone reads leaves first, so that a step's block
// tables, lengths and instructions stay.
__device__ __forceinline__ uint64_t l2_policy(bool once) {
  uint64_t p;
  if (once)
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// 4-D tiled load (c0 innermost), completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* tm, uint64_t* bar,
                                            int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %3, %3, %4}], [%2], %5;" ::"r"(ptx::smem_u32(dst)),
      "l"(tm), "r"(ptx::smem_u32(bar)), "r"(0), "r"(c3), "l"(policy)
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

// Brings in the K and V rows of key tiles: a box per page (or per 128 rows of a
// larger one).  The page ids of 32 boxes are looked up at once, a lane each, and
// the next 32 ahead of their use.  Pages that no row sees are not touched.  A
// page that is missing is asked for past the cache's end, where the tensor map
// reads zeros.  One warp; the tiles of a segment in their order.
template <int D>
struct TileLoader {
  int page, lg_page, box, boxes, per;
  uint64_t policy;
  int now;   // where this lane's box starts in the cache, in groups of eight rows,
             // in this batch of `per` tiles; -1: not needed
  int next;  // its page's id in the next batch, as the table has it, if it is needed
  bool next_seen;
  __device__ __forceinline__ explicit TileLoader(const AttnParams& P)
      : page(P.kv.page_size),
        lg_page(P.lg_page),
        box(P.box),
        boxes(kKeys / box),
        per(32 / boxes),
        next(0) {}
  // This lane's box of the batch from tile i0: whether some row sees it, its page's
  // id as the table has it (a load that nothing here waits for; any value of the
  // type may come), and where it starts.
  __device__ __forceinline__ int first_place(const Segment& g, int i0) const {
    const int lane = threadIdx.x & 31;
    return (g.first + i0 + lane / boxes) * kKeys + (lane & (boxes - 1)) * box;
  }
  __device__ __forceinline__ int first_key(const Segment& g, int i0) const {
    const int v = first_place(g, i0);
    return v < g.t.sink_places ? v : window_key(g.t, v);
  }
  __device__ __forceinline__ int fetch(const AttnParams& P, const Segment& g, int i0,
                                       bool& seen) const {
    const int key0 = first_key(g, i0);
    seen = i0 + (threadIdx.x & 31) / boxes < g.n &&
           ((key0 <= g.t.vis_hi && key0 + box - 1 >= g.t.vis_lo) ||
            first_place(g, i0) < g.t.n_sink);
    return seen ? P.kv.block_table[static_cast<int64_t>(g.table_row) * P.kv.max_pages +
                                   (key0 >> lg_page)]
                : 0;
  }
  __device__ __forceinline__ int place(const AttnParams& P, const Segment& g, int i0, int id,
                                       bool seen) const {
    if (!seen) return -1;
    if (id < 0 || id >= P.kv.n_pages) {
      flag_error(P.err, LORA_DEVERR_BAD_PAGE);
      return P.kv.n_pages * P.kv.n_kv_heads * (page / 8);
    }
    return (id * P.kv.n_kv_heads + g.head) * (page / 8) + (first_key(g, i0) & (page - 1)) / 8;
  }
  __device__ __forceinline__ void begin(const AttnParams& P, const Segment& g) {
    policy = l2_policy(g.once != 0);
    bool seen;
    const int id = fetch(P, g, 0, seen);
    next_seen = false;
    if (g.n > per) next = fetch(P, g, per, next_seen);
    now = place(P, g, 0, id, seen);
  }
  // The place of this lane's box of tile i (lanes below `boxes`).
  __device__ __forceinline__ int at(const AttnParams& P, const Segment& g, int i) {
    const int k = i % per;
    if (k == 0 && i > 0) {
      now = place(P, g, i, next, next_seen);
      next_seen = false;
      if (i + per < g.n) next = fetch(P, g, i + per, next_seen);
    }
    const int lane = threadIdx.x & 31;
    const int x = __shfl_sync(0xffffffffu, now, k * boxes + (lane & (boxes - 1)));
    return lane < boxes ? x : -1;
  }
  __device__ __forceinline__ uint32_t bytes(int at) const {  // of all lanes' boxes
    return __popc(__ballot_sync(0xffffffffu, at >= 0)) * box_bytes();
  }
  __device__ __forceinline__ uint32_t box_bytes() const { return static_cast<uint32_t>(box) * D * 2; }
  __device__ __forceinline__ void load(const CUtensorMap* tm, uint64_t* full, uint8_t* dst, int at,
                                       uint32_t all) const {
    const int lane = threadIdx.x & 31;
    if (lane == 0) ptx::mbar_arrive_expect_tx(full, all);
    __syncwarp();
    if (at >= 0) tma_load_4d(dst + lane * box_bytes(), tm, full, at, policy);
  }
};

// Writes a finished row (token t, query head h; sums of exponentials `sum` at the
// maximum m, log2 units), eight values at a time: x / sum.  The prefix phase
// keeps it in fp32 with its log-sum-exp; otherwise it is joined with that part,
// if there is one, and rounded to out.
template <int D>
struct RowWriter {
  float own, other;  // factors of this result and of the prior part
  bf16* out;
  float* prior;
  bool to_prior, join;
  __device__ __forceinline__ RowWriter(const AttnParams& P, int shared, int64_t t, int h,
                                       bool in_use, float m, float sum) {
    to_prior = P.groups_phase;
    join = !to_prior && shared;
    own = sum > 0.f ? 1.f / sum : 0.f;
    other = 0.f;
    out = P.out + t * P.out_stride + h * D;
    const int64_t at = t * P.n_q_heads + h;
    prior = P.prior + at * D;
    if ((to_prior || join) && in_use) {
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
  // Sixteen values, in one 32-byte store where `out` allows it.
  __device__ __forceinline__ void write16(int d, const float* x) const {
    if (to_prior || join || (reinterpret_cast<uintptr_t>(out) & 31) != 0) {
      write8(d, x);
      write8(d + 8, x + 8);
      return;
    }
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = pack_bf16x2(x[2 * i] * own, x[2 * i + 1] * own);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + d),
                 "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]),
                 "r"(u[7])
                 : "memory");
  }
};

// The slot of the item's c-th part.
__device__ __forceinline__ int64_t part_slot(const Segment& g, int c) {
  return static_cast<int64_t>(g.cta0 + c) * 2 + (c == 0 ? 1 : 0);
}

// Threads of named barrier `bar` (cnt of them) have written this CTA's part:
// is it the last of the item (or of its half)?  Leaves the counter at zero.
__device__ __forceinline__ bool last_to_arrive(const AttnParams& P, const Segment& g, int half,
                                               bool leader, int* flag, int bar, int cnt) {
  uint32_t* count = P.count + g.cta0 * 2 + half;
  __threadfence();
  named_bar(bar, cnt);
  if (leader) {
    const uint32_t before = atomicAdd(count, 1u);
    *flag = before + 1 == static_cast<uint32_t>(g.parts) ? 1 : 0;
    if (*flag) *count = 0;
    __threadfence();
  }
  named_bar(bar, cnt);
  __threadfence();
  return *flag != 0;
}

}  // namespace lora
