// Parts that the attention kernels' warps share: bounded waits, the TMA
// producer, values that no row sees, and writing, splitting and joining
// results.
#pragma once

#include "attn.cuh"
#include "fp8.cuh"
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
// The same with rows of `span` bytes, which the swizzle spans (128, 64, or 0: none).
__host__ __device__ constexpr uint32_t desc_hi_span(uint32_t sbo_bytes, uint32_t span) {
  return ((sbo_bytes >> 4) & 0x3FFFu) | (1u << 14) | ((span == 128 ? 2u : span == 64 ? 4u : 0u) << 29);
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
// The same of 8-bit floating types.
__device__ __forceinline__ void mma_ss_8bit(uint32_t d, uint32_t a_lo, uint32_t a_hi,
                                            uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d),
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
// reads zeros.  One warp; the tiles of a segment in their order.  kElem: bytes of
// a value.
template <int D, int kElem = 2>
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
  // The segment's first page ids, on their way: place(P, g, 0, id, seen) has to become `now`.
  __device__ __forceinline__ int ask(const AttnParams& P, const Segment& g, bool& seen) {
    policy = l2_policy(g.once != 0);
    const int id = fetch(P, g, 0, seen);
    next_seen = false;
    if (g.n > per) next = fetch(P, g, per, next_seen);
    return id;
  }
  __device__ __forceinline__ void begin(const AttnParams& P, const Segment& g) {
    bool seen;
    const int id = ask(P, g, seen);
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
  __device__ __forceinline__ uint32_t box_bytes() const { return static_cast<uint32_t>(box) * D * kElem; }
  __device__ __forceinline__ void load(const CUtensorMap* tm, uint64_t* full, uint8_t* dst, int at,
                                       uint32_t all) const {
    const int lane = threadIdx.x & 31;
    if (lane == 0) ptx::mbar_arrive_expect_tx(full, all);
    __syncwarp();
    if (at >= 0) tma_load_4d(dst + lane * box_bytes(), tm, full, at, policy);
  }
};

// Scales of the 8-bit cache's key tiles, a batch of P.scale_tiles of them at a time, ahead of
// their use.  Batch n of the CTA lies in tiles 4 (n % kBatches) and on.
template <int kBatches>
struct ScaleRing {
  float k[4 * kBatches][16];    // of a tile's blocks of keys
  uint8_t v[4 * kBatches][16];  // bytes of its blocks of values
  int top[4 * kBatches];        // the largest of them since the segment's first tile
  uint64_t full[kBatches], empty[kBatches];
};
// One thread; `readers` arrivals free a batch.
template <int kBatches>
__device__ __forceinline__ void init_scales(ScaleRing<kBatches>& S, int readers) {
  for (int i = 0; i < kBatches; ++i) {
    ptx::mbar_init(&S.full[i], 1);
    ptx::mbar_init(&S.empty[i], readers);
  }
}
// A reader's way through them: of(i) before tile i of segment g, done(i) after it (all lanes).
struct ScaleReader {
  int lg;  // log2 of a batch' tiles
  __device__ __forceinline__ explicit ScaleReader(const AttnParams& P) : lg(P.scale_tiles == 2 ? 1 : 2) {}
  __device__ __forceinline__ int batch(const Segment& g, int i) const { return g.batch0 + (i >> lg); }
  template <int kBatches>
  __device__ __forceinline__ int of(ScaleRing<kBatches>& S, const Segment& g, int i, volatile int* abort) const {
    const int n = batch(g, i), in = i & ((1 << lg) - 1);
    if (in == 0) wait_quiet(&S.full[n % kBatches], (n / kBatches) & 1, abort);
    return n % kBatches * 4 + in;
  }
  // `times`: for how many warps
  template <int kBatches>
  __device__ __forceinline__ void done(ScaleRing<kBatches>& S, const Segment& g, int i, int times = 1) const {
    if ((i & ((1 << lg) - 1)) != (1 << lg) - 1 && i != g.n - 1) return;
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
      for (int k = 0; k < times; ++k) ptx::mbar_arrive(&S.empty[batch(g, i) % kBatches]);
  }
};
// Looks them up, one warp: a lane to a block, as many tiles at once as 32 lanes have blocks
// of, the next ones' page ids on their way beside them.  Scales of blocks that no row sees
// are not read: 1 for keys, and for values a byte that leaves `top` where it is.
struct ScaleFinder {
  int block, lg_block, per_tile, at_once;
  int mine, b;    // this lane's tile of a batch, and its block there
  int id, key0, top;
  bool seen;
  __device__ __forceinline__ explicit ScaleFinder(const AttnParams& P)
      : block(min(P.kv.page_size, kScaleBlock)),
        lg_block(block == 8 ? 3 : 4),
        per_tile(kKeys / block),
        at_once(P.scale_tiles),
        mine((threadIdx.x & 31) / per_tile),
        b((threadIdx.x & 31) % per_tile) {}
  __device__ __forceinline__ void fetch(const AttnParams& P, const Segment& g, int i0) {
    const int v = (g.first + i0 + mine) * kKeys + b * block;
    key0 = v < g.t.sink_places ? v : window_key(g.t, v);
    seen = i0 + mine < g.n &&
           ((key0 <= g.t.vis_hi && key0 + block - 1 >= g.t.vis_lo) || v < g.t.n_sink);
    if (seen)
      id = P.kv.block_table[static_cast<int64_t>(g.table_row) * P.kv.max_pages + (key0 >> P.lg_page)];
  }
  __device__ __forceinline__ void begin(const AttnParams& P, const Segment& g) {
    top = 0;
    fetch(P, g, 0);
  }
  // Tiles i0 .. i0 + at_once - 1 of the segment; false once a wait of the CTA gave up.
  template <int kBatches>
  __device__ __forceinline__ bool fill(const AttnParams& P, ScaleRing<kBatches>& S,
                                       const Segment& g, int i0, volatile int* abort) {
    const int lane = threadIdx.x & 31;
    int kb = 127, vb = 1;
    if (seen && id >= 0 && id < P.kv.n_pages) {
      const int64_t at =
          (static_cast<int64_t>(id) * P.kv.n_kv_heads + g.head) * (P.kv.page_size >> lg_block) +
          ((key0 & (P.kv.page_size - 1)) >> lg_block);
      kb = scale_read(P.k_scale[at]);
      vb = scale_read(P.v_scale[at]);
    }
    if (i0 + at_once < g.n) fetch(P, g, i0 + at_once);
    const int n = min(at_once, g.n - i0), batch = g.batch0 + i0 / at_once;
    const int slot = batch % kBatches;
    if (batch >= kBatches && !wait_all(&S.empty[slot], ((batch / kBatches) & 1) ^ 1, abort))
      return false;
    if (mine < n) {
      S.k[slot * 4 + mine][b] = scale_of(kb);
      S.v[slot * 4 + mine][b] = static_cast<uint8_t>(vb);
    }
    // the largest so far, tile by tile
    for (int i = 0; i < n; ++i) {
      top = max(top, __reduce_max_sync(0xffffffffu, mine == i ? vb : 0));
      if (lane == 0) S.top[slot * 4 + i] = top;
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.full[slot]);
    return true;
  }
};

// The whole of a warp's work: scales of all tiles of the segments in `ring`, to the first end.
template <int kBatches>
__device__ __forceinline__ void run_scales(const AttnParams& P, ScaleRing<kBatches>& S,
                                           const Segment* ring, int ring_size, uint64_t* seg_full,
                                           uint64_t* seg_empty, volatile int* abort) {
  ScaleFinder find(P);
  bool ok = true;
  for (int sg = 0; ok; ++sg) {
    ok = wait_all(&seg_full[sg % ring_size], (sg / ring_size) & 1, abort);
    if (!ok) break;
    const Segment& g = ring[sg % ring_size];
    if (g.n == 0) break;
    find.begin(P, g);
    for (int i = 0; i < g.n && ok; i += find.at_once) ok = find.fill(P, S, g, i, abort);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&seg_empty[sg % ring_size]);
  }
}

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

// Of a row's weights over an 8-bit cache, whose values lack a power of two, their `unit`: the
// weights' sum l over a part of the keys is brought into [1, 2) and the maximum moved with it, so
// that a part is as large as a value, not as all weights together, which the ends of fp32 would
// not hold.  `down`: what l and the values are to be multiplied with, `up` its inverse, in log2.
struct PartScale {
  float down, up;
  __device__ __forceinline__ explicit PartScale(float l) {
    const int e = l > 0.f ? min(max(static_cast<int>(__float_as_uint(l) >> 23), 1), 253) : 127;
    down = scale_of(254 - e);
    up = static_cast<float>(e - 127);
  }
};
// A whole row's, where its factor is 1 / l: a small unit is not made part of it, since the two
// together would be below the normal numbers, and so lose bits, where a result is not.
struct RowUnit {
  float first, factor;  // of the values, and of 1 / l
  __device__ __forceinline__ explicit RowUnit(float unit) {
    const bool small = unit < 0x1p-40f;
    first = small ? unit : 1.f;
    factor = small ? 1.f : unit;
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

// The end of an item, or of this CTA's part of it, in the kernels that have few rows
// to a key head (A in a row tile): 128 threads of named barrier `bar` write the rows from
// `stage` [A][D], maxima m [A] (log2 units) and the four warps' sums red_sum [A], joined with
// the parts of other CTAs by the last to arrive.  kUnits: the rows are to be multiplied with `unit`.
template <int D, int A, bool kUnits = false>
__device__ __forceinline__ void finish_rows(const AttnParams& P, const Segment& g,
                                            const float* stage, const float* m,
                                            const float4* red_sum, int tid, int* last, int bar,
                                            float unit = 1.f) {
  float2* ml = reinterpret_cast<float2*>(P.part_ml);
  const int vectors = g.t.n_rows * (D / 8);
  bool write = true;
  if (g.parts > 1) {
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + g.slot;
#pragma unroll 1
    for (int x = tid; x < vectors; x += 128) {
      const int n = x / (D / 8), k = x % (D / 8) * 8;
      const float4 r = red_sum[n];
      if constexpr (kUnits) {
        const float l = r.x + r.y + r.z + r.w;
        const PartScale by(l);
        float o[8];
        load8(stage + n * D + k, o);
#pragma unroll
        for (int y = 0; y < 8; ++y) o[y] = o[y] * by.down * unit;
        store8(P.part + (slot * A + n) * D + k, o);
        if (k == 0) ml[slot * A + n] = make_float2(m[n] + by.up, l * by.down);
      } else {
        store8(P.part + (slot * A + n) * D + k,
               *reinterpret_cast<const float(*)[8]>(stage + n * D + k));
        if (k == 0) ml[slot * A + n] = make_float2(m[n], r.x + r.y + r.z + r.w);
      }
    }
    write = last_to_arrive(P, g, 0, tid == 0, last, bar, 128);
  }
#pragma unroll 1
  for (int x = write ? tid : vectors; x < vectors; x += 128) {
    const int n = x / (D / 8), k = x % (D / 8) * 8;
    float o[8], top, sum;
    if (g.parts == 1) {
      const float4 r = red_sum[n];
      top = m[n];
      sum = r.x + r.y + r.z + r.w;
      load8(stage + n * D + k, o);
    } else {
      // all parts, in their order
      top = -INFINITY, sum = 0.f;
#pragma unroll 4
      for (int q = 0; q < g.parts; ++q)
        top = fmaxf(top, __ldcg(&ml[part_slot(g, q) * A + n].x));
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] = 0.f;
#pragma unroll 4
      for (int q = 0; q < g.parts; ++q) {
        const float2 v = __ldcg(&ml[part_slot(g, q) * A + n]);
        const float4* from =
            reinterpret_cast<const float4*>(P.part + (part_slot(g, q) * A + n) * D + k);
        const float4 a = __ldcg(from), b = __ldcg(from + 1);
        const float f = top == -INFINITY ? 0.f : exp2_fast(v.x - top);
        sum += f * v.y;
        o[0] += f * a.x; o[1] += f * a.y; o[2] += f * a.z; o[3] += f * a.w;
        o[4] += f * b.x; o[5] += f * b.y; o[6] += f * b.z; o[7] += f * b.w;
      }
    }
    const int r = g.t.row0 + n, tok = P.by_group(r);
    RowWriter<D> out(P, g.shared, g.tok0 + tok, g.head * P.group + r - tok * P.group, true,
                     top, sum);
    if (kUnits && g.parts == 1) {
      const RowUnit by(unit);
      out.own *= by.factor;
#pragma unroll
      for (int y = 0; y < 8; ++y) o[y] *= by.first;
    }
    out.write8(k, o);
  }
}

}  // namespace lora
