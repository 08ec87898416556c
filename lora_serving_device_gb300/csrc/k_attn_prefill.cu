// Attention over the paged cache for many rows per key head: prompts, chunks
// of prompts and the tokens of a prefix group (lora_attn_paged and the prefix
// phase of lora_attn_prefix).
//
// Mathematics, per item (two halves of up to 128 rows of one key head) and
// key tile of 128 keys, for each half:
//   S  = Q K^T             [128 rows, 128 keys]   tcgen05, fp32 in tensor memory
//   P  = 2^(S c - m)       c = scale log2(e), m the row's reference maximum
//   l += row sums of P
//   O += P V               [128 rows, D]          tcgen05, P bf16 from tensor memory
// m is moved (and l, O scaled) only where a score exceeds it by more than 8 in
// log2 units, so the usual tile leaves O alone.  P is rounded to bf16, the type
// the MMA takes beside V; l sums the unrounded values in fp32.
//
// Bound by the tensor cores: 4 x 128 x 128 x D operations a half and tile.
// The two halves alternate: while one half's softmax runs on its warpgroup,
// the tensor cores work for the other.  A softmax thread owns one row (a
// tensor-memory lane), so maximum and sum need no exchange; P overwrites S in
// tensor memory and never passes through shared memory.  Rows are (token,
// query head of the key head), so all query heads of a key head share each
// K and V tile; a half holds whole tokens, which lets TMA fetch Q too.
//
// Measured: a prompt of 8192, 32 / 8 heads of 128: 373 us, 1475 TFLOP/s (0.76 of
// the measured burst rate, 0.83 of the sustained one); 348 us in the first
// moments on a cool card.  The tensor pipe is active for 69% of the cycles (345
// us under the profiler), the exponentials' for 35%.  What is
// left is the way from scores to weights and back: S and P share tensor
// memory, which the two halves' S and O fill, so a half's next scores wait for
// its last product.  P handed over as a whole costs 3%, in quarters 6%, after
// three quarters 4%; two threads to a row, with a vote a tile, 14%.
// Chunks with a window of 1024 (9.1 tiles an item): 117 us, 46% of the cycles.
// The roles' loops are kept short.  With more instructions in them a warp waited
// 0.61 cycles an issue for its instruction (now 0.39): those chunks took 140 us,
// a prompt of 4000, 64 / 8 heads of 64, 182 where it takes 160 (the operations of
// its product alone: 67 us; it takes twice the exponentials an operation).
//
// Warps: 0-3 softmax of half 0, 4-7 of half 1 (and their results), 8 schedule
// and TMA, 9 MMA issue.  Every wait is bounded; on timeout the kernel raises
// LORA_DEVERR_TIMEOUT.
#include <cudaTypedefs.h>

#include "attn_rows.cuh"

namespace lora {
namespace {

// Three warpgroups: the softmax threads hold a row of 128 scores each and take
// registers from the third, of which two warps work.  192 x 256 + 120 x 128 is
// within the launch's 168 x 384.
constexpr int kThreads = 384;
constexpr int kRegsMost = 192, kRegsLeast = 120;
constexpr int kRing = 4;     // segments that the producer may run ahead

template <int D>
struct Lay {
  static constexpr uint32_t kTile = kKeys * D * 2;  // K or V of a tile, Q of a half
  static constexpr int kSlots = D == 128 ? 5 : 10;  // K and V tiles in flight
  static constexpr uint32_t oQ = kSlots * kTile;
  static constexpr uint32_t oMisc = oQ + 2 * kTile;
};

template <int kSlots>
struct Misc {
  Segment ring[kRing];
  uint64_t full[kSlots], empty[kSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2], o_empty[2];
  uint64_t seg_full[kRing], seg_empty[kRing];
  uint32_t tmem;
  int abort;
  int last[2];
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const AttnParams P) {
  using La = Lay<D>;
  constexpr int kSlots = La::kSlots;
  using Mi = Misc<kSlots>;
  constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(kHalf, kKeys, false, false);
  constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kHalf, D, false, true);
  constexpr uint32_t kGroupBytes = (D / 64) * 1024;  // eight keys

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Mi& M = *reinterpret_cast<Mi*>(smem + La::oMisc);
  volatile int* abort_f = &M.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half_rows = P.rows / 2;  // rows of a half that are in use

  if (tid == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&M.full[i], 1);
      ptx::mbar_init(&M.empty[i], 1);
    }
    for (int h = 0; h < 2; ++h) {
      ptx::mbar_init(&M.q_full[h], 1);
      ptx::mbar_init(&M.q_empty[h], 1);
      ptx::mbar_init(&M.s_full[h], 1);
      ptx::mbar_init(&M.p_half[h], 4);
      ptx::mbar_init(&M.p_full[h], 4);
      ptx::mbar_init(&M.o_done[h], 1);
      ptx::mbar_init(&M.o_empty[h], 4);
    }
    for (int i = 0; i < kRing; ++i) {
      ptx::mbar_init(&M.seg_full[i], 1);
      ptx::mbar_init(&M.seg_empty[i], 9);
    }
    M.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(&M.tmem, 512);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  // (the next grid may not start early: its launch slows this one's last CTAs,
  // which join parts, by more than its prologue takes)
  pdl_wait();
  // the tiles' memory holds the problems' sizes until the first load
  size_problems(P, reinterpret_cast<ProblemSize*>(smem));
  __syncthreads();
  size_long_problems(P, reinterpret_cast<ProblemSize*>(smem));
  ptx::fence_proxy_async_smem();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = M.tmem;  // S (and P) of half h at h * 128, O at 256 + h * 128

  // (each role's branch begins with its own split, so that the compiler knows
  // the number of registers on every path)
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLeast));
  if (warp == 8) {
    // ---------------- schedule and TMA ----------------------------------
    Walker walk;
    walk.start(P, reinterpret_cast<ProblemSize*>(smem));
    ptx::fence_proxy_async_smem();
    __syncwarp();
    TileLoader<D> load(P);
    int n = 0;              // tiles brought in: K in slot 2n, V in slot 2n + 1
    int q_use[2] = {0, 0};  // segments of each half
    bool ok = true;
    SplitItem mine = {};
    for (int sg = 0; ok; ++sg) {
      const Segment g = walk.next(P);
      if (sg >= kRing)
        ok = wait_all(&M.seg_empty[sg % kRing], ((sg / kRing) & 1) ^ 1, abort_f);
      if (!ok) break;
      if (lane == 0) {
        M.ring[sg % kRing] = g;
        ptx::mbar_arrive(&M.seg_full[sg % kRing]);
      }
      __syncwarp();
      if (g.n == 0) break;
      load.begin(P, g);
      if (P.join_after && g.parts > 1 && g.cta0 == blockIdx.x)
        mine = {g.parts, g.tok0, g.t.row0, g.t.n_rows, g.head, g.shared, {0, 0}};
      for (int h = 0; h < 2 && ok; ++h) {
        if (g.t.n_rows <= h * half_rows) break;
        if (q_use[h] > 0) ok = wait_all(&M.q_empty[h], (q_use[h] - 1) & 1, abort_f);
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&M.q_full[h], half_rows * D * 2);
          for (int x = 0; x < D / 64; ++x)
            tma_load_rows(smem + La::oQ + h * La::kTile + x * (kHalf * 128), &tm_q, &M.q_full[h],
                          g.head * P.group, g.tok0 + P.by_group(g.t.row0 + h * half_rows), x);
        }
        ++q_use[h];
      }
      __syncwarp();
      for (int i = 0; i < g.n && ok; ++i, ++n) {
        const int at = load.at(P, g, i);
        const uint32_t bytes = load.bytes(at);
        for (int v = 0; v < 2; ++v) {
          const int k = 2 * n + v, st = k % kSlots;
          if (k >= kSlots) ok = wait_all(&M.empty[st], ((k / kSlots) & 1) ^ 1, abort_f);
          if (!ok) break;
          load.load(v ? &tm_v : &tm_k, &M.full[st], smem + st * La::kTile, at, bytes);
        }
      }
    }
    if (P.join_after && lane == 0) P.split[blockIdx.x] = mine;
    if (!ok) {
      // gave up: what is on its way into shared memory has to land first
      int none = 0;
      for (int h = 0; h < 2; ++h)
        if (q_use[h] > 0)
          ptx::mbar_wait_bounded(&M.q_full[h], (q_use[h] - 1) & 1, &none, kAttnWaitNs / 8);
      for (int k = 2 * n > kSlots ? 2 * n - kSlots : 0; k < 2 * n; ++k)
        ptx::mbar_wait_bounded(&M.full[k % kSlots], (k / kSlots) & 1, &none, kAttnWaitNs / 8);
    }
  } else if (warp == 9) {
    // ---------------- MMA issue ------------------------------------------
    // One thread: P V of tile n and Q K^T of tile n + 1, half by half, so that
    // the tensor cores have the other half's work while a softmax runs.
    if (elect_one()) {
      const uint32_t slots = desc_lo(ptx::smem_u32(smem), 0);
      // A bit for each half: parities of its Qs, of its tiles' P and of its O, and
      // whether it has had a segment.
      uint32_t q_par = 0, p_par = 0, o_par = 0, begun = 0;
      auto issue_qk = [&](bool first, bool last, int n, int h, bool frees) {
        if (first) {
          wait_quiet(&M.q_full[h], (q_par >> h) & 1, abort_f);
          q_par ^= 1u << h;
        }
        const int k = 2 * n, st = k % kSlots;
        wait_quiet(&M.full[st], (k / kSlots) & 1, abort_f);
        ptx::tc_fence_after();
        const uint32_t qa = desc_lo(ptx::smem_u32(smem + La::oQ + h * La::kTile), 16);
        const uint32_t ka = slots + st * (La::kTile / 16) + (1u << 16);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)  // Q: [64-value half of a head][128 rows][64]
          mma_ss(tmem + h * 128, qa + ((ks / 4) * (kHalf * 128) + (ks % 4) * 32) / 16,
                 desc_hi(1024), ka + ((ks / 4) * 1024 + (ks % 4) * 32) / 16, desc_hi(kGroupBytes),
                 kIdescQK, ks > 0 ? 1u : 0u);
        ptx::mma_commit(&M.s_full[h]);
        if (frees) ptx::mma_commit(&M.empty[st]);
        if (last) ptx::mma_commit(&M.q_empty[h]);
      };
      auto issue_pv = [&](bool first, int n, int h, bool frees) {
        const int k = 2 * n + 1, st = k % kSlots;
        const uint32_t va = slots + st * (La::kTile / 16) + ((1024u / 16) << 16);
        if (h == 0) wait_quiet(&M.full[st], (k / kSlots) & 1, abort_f);
        if (first) {
          // the half's previous segment has been read out of O
          if ((begun >> h) & 1) {
            wait_quiet(&M.o_empty[h], (o_par >> h) & 1, abort_f);
            o_par ^= 1u << h;
          }
          begun |= 1u << h;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          wait_quiet(x ? &M.p_full[h] : &M.p_half[h], (p_par >> h) & 1, abort_f);
          ptx::tc_fence_after();
#pragma unroll
          for (int ks = 4 * x; ks < 4 * x + 4; ++ks)
            mma_ts(tmem + 256 + h * 128, tmem + h * 128 + ks * 8,
                   va + ks * 2 * kGroupBytes / 16, desc_hi(kGroupBytes), kIdescPV,
                   ks > 0 || !first ? 1u : 0u);
        }
        ptx::mma_commit(&M.o_done[h]);
        if (frees) ptx::mma_commit(&M.empty[st]);
        p_par ^= 1u << h;
      };
      int sg = -1, left = 0;  // the segment of tile n, and its key tiles to go
      bool two = false, first = false;
#pragma unroll 1
      for (int n = -1; !*abort_f; ++n) {
        int next = left - 1;
        bool next_two = two, next_first = false;
        if (next <= 0) {  // the next tile is of the next segment
          wait_quiet(&M.seg_full[(sg + 1) % kRing], ((sg + 1) / kRing) & 1, abort_f);
          next = M.ring[(sg + 1) % kRing].n;
          next_two = M.ring[(sg + 1) % kRing].t.n_rows > half_rows;
          next_first = true;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (left > 0 && h <= two) issue_pv(first, n, h, h == two);
          if (next > 0 && h <= next_two) issue_qk(next_first, next == 1, n + 1, h, h == next_two);
        }
        if (next_first) {
          if (sg >= 0) ptx::mbar_arrive(&M.seg_empty[sg % kRing]);
          ++sg;
        }
        if (next <= 0) break;
        left = next;
        two = next_two;
        first = next_first;
      }
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMost));
    // ---------------- softmax and results ---------------------------------
    const int h = warp >> 2, w = warp & 3;
    const int row = w * 32 + lane;  // of the half, and the TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    const uint32_t tm_s = tmem + lanes + h * 128, tm_o = tmem + lanes + 256 + h * 128;
    const float c = P.scale_log2;
    const int bar = 1 + h;
    int tile = 0;  // tiles of this half so far
    // The warpgroup's four warps meet at barriers: after a wait that gave up
    // they run on (every later wait returns at once) to the vote.
    for (int sg = 0;; ++sg) {
      wait_quiet(&M.seg_full[sg % kRing], (sg / kRing) & 1, abort_f);
      if (named_any(bar, 128, *abort_f != 0)) break;
      const Segment g = M.ring[sg % kRing];
      if (g.n == 0) break;
      const int n_rows = min(g.t.n_rows - h * half_rows, half_rows);  // of this half
      if (n_rows <= 0) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&M.seg_empty[sg % kRing]);
        continue;
      }
      // rows past the last copy the first one
      const bool mine = row < n_rows;
      const int in_prob = g.t.row0 + h * half_rows + (mine ? row : 0);
      const int tok = P.by_group(in_prob), head = g.head * P.group + in_prob - tok * P.group;
      const int pos = g.base + tok;
      const int hi = P.groups_phase ? g.t.vis_hi : min(pos, g.t.vis_hi);
      const int lo = P.groups_phase ? 0 : max(window_first(P, pos), g.k_lo);
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int i = 0; i < g.n; ++i, ++tile) {
        const int v0 = (g.first + i) * kKeys, key0 = window_key(g.t, v0);  // place, key
        wait_quiet(&M.s_full[h], tile & 1, abort_f);
        __syncwarp();
        ptx::tc_fence_after();
        float s[kKeys];
#pragma unroll
        for (int k = 0; k < kKeys; k += 32)
          ptx::tmem_ld32(tm_s + k, *reinterpret_cast<uint32_t(*)[32]>(s + k));
        ptx::tmem_ld_wait();
        mask_scores(tm_s, key0, hi, lo, min(g.t.n_sink, hi + 1) - v0, s);
        float mx = max3(s[0], s[1], s[2]), my = max3(s[3], s[4], s[5]);
        float mz = max3(s[6], s[7], s[8]), mw = max3(s[9], s[10], s[11]);
#pragma unroll
        for (int k = 12; k + 7 < kKeys; k += 8) {
          mx = max3(mx, s[k], s[k + 1]);
          my = max3(my, s[k + 2], s[k + 3]);
          mz = max3(mz, s[k + 4], s[k + 5]);
          mw = max3(mw, s[k + 6], s[k + 7]);
        }
        mx = max3(mx, s[kKeys - 4], s[kKeys - 3]);
        my = max3(my, s[kKeys - 2], s[kKeys - 1]);
        mx = max3(mx, my, fmaxf(mz, mw)) * c;
        // (rows that are not in use hold anything: they have no say)
        if (__any_sync(0xffffffffu, mine && mx > m + 8.f)) {
          const float now = fmaxf(m, mx);
          const float f = m == -INFINITY ? 0.f : exp2_fast(m - now);
          m = now;
          l *= f;
          if (i > 0) {
            wait_quiet(&M.o_done[h], (tile - 1) & 1, abort_f);
            __syncwarp();
            ptx::tc_fence_after();
            scale_result<D>(tm_o, f);
          }
        }
        if (h == 0 && tile_has_unseen(g.t, v0)) {
          // (half 0 takes part in every tile, and its P V is issued first)
          const int k = 2 * tile + 1;
          wait_quiet(&M.full[k % kSlots], (k / kSlots) & 1, abort_f);
          zero_unseen_value<D>(g.t, v0, row, smem + (k % kSlots) * La::kTile);
          ptx::fence_proxy_async_smem();
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        const uint64_t c2 = pack2(c, c), neg2 = pack2(neg, neg);
        uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
        for (int k = 0; k < kKeys; k += 32) {
          uint32_t p[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float a, b;
            unpack2(fma2(pack2(s[k + 2 * x], s[k + 2 * x + 1]), c2, neg2), &a, &b);
            a = exp2_fast(a);
            b = exp2_fast(b);
            if (x & 1)
              sum1 = add2(sum1, pack2(a, b));
            else
              sum0 = add2(sum0, pack2(a, b));
            p[x] = pack_bf16x2(a, b);
          }
          ptx::tmem_st16(tm_s + k / 2, p);
          if (k == 32 || k == 96) {
            // each half of the keys goes to the MMA as soon as it is there
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(k == 32 ? &M.p_half[h] : &M.p_full[h]);
          }
        }
        float a, b;
        unpack2(add2(sum0, sum1), &a, &b);
        l += a + b;
      }

      // ---- the item, or this CTA's part of it, is done
      finish_half<D>(P, g, h, row, mine, g.tok0 + tok, head, m, l, 1.f, tm_o, &M.o_done[h],
                     (tile - 1) & 1, abort_f, &M.o_empty[h], &M.seg_empty[sg % kRing], &M.last[h], bar);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && *abort_f) flag_error(P.err, LORA_DEVERR_TIMEOUT);
}

// Joins the parts of the items that several CTAs shared, where there can be
// many of each.  The work is cut into pieces of 32 rows and half the columns;
// each block looks up the split items and takes every kJoinBlocks-th piece.
// A lane is a row; each warp adds up its columns over the parts, so that all
// reads are whole lines, and the rows are written from shared memory.
constexpr int kJoinBlocks = 4 * kDecodeScheduleCtas;

template <int D>
__device__ __forceinline__ void join_piece(const AttnParams& P, const SplitItem& it, int c, int h,
                                           int row0, int z, float2 (*fac)[32],
                                           float4 (*rows)[D / 8 + 1], float* top_s, float* sum_s) {
  constexpr int kCols = D / 2, kPer = kCols / 4 / 8;  // vectors of a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half_rows = P.rows / 2, row = row0 + lane;
  const bool used = row < half_rows && h * half_rows + row < it.n_rows;
  auto slot = [&](int q) { return static_cast<int64_t>(c + q) * 2 + (q == 0 ? 1 : 0); };
  const float2* ml = reinterpret_cast<const float2*>(P.part_ml) + h * kHalf + row;
  const int k0 = z * (kCols / 4) + warp * kPer;
  auto value = [&](int q, int x) { return part_row<D>(P, slot(q), h, row)[(k0 + x) * kHalf]; };
  // the first parts' values are on their way beside the maxima and sums
  constexpr int kAhead = 8;
  float4 v[kAhead][kPer];
#pragma unroll
  for (int q = 0; q < kAhead; ++q)
#pragma unroll
    for (int x = 0; x < kPer; ++x) v[q][x] = q < it.parts ? value(q, x) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int q = warp; q < it.parts; q += 8)
    fac[q][lane] = used ? ml[slot(q) * 2 * kHalf] : make_float2(-INFINITY, 0.f);
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int q = 0; q < it.parts; ++q) top = fmaxf(top, fac[q][lane].x);
  const float ref = top == -INFINITY ? 0.f : top;
  float4 o[kPer];
#pragma unroll
  for (int x = 0; x < kPer; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int q0 = 0; q0 < it.parts; q0 += kAhead) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (q0 + q >= it.parts) break;
      const float2 z = fac[q0 + q][lane];
      const float f = exp2f(z.x - ref);
      sum += f * z.y;
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        o[x].x += f * v[q][x].x;
        o[x].y += f * v[q][x].y;
        o[x].z += f * v[q][x].z;
        o[x].w += f * v[q][x].w;
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
#pragma unroll
      for (int x = 0; x < kPer; ++x)
        if (q0 + kAhead + q < it.parts) v[q][x] = value(q0 + kAhead + q, x);
  }
  if (warp == 0) {
    top_s[lane] = top;
    sum_s[lane] = sum;
  }
#pragma unroll
  for (int x = 0; x < kPer; ++x) rows[lane][warp * kPer + x] = o[x];
  __syncthreads();
  for (int x = threadIdx.x; x < 32 * (kCols / 8); x += 256) {
    const int r = x / (kCols / 8), k = x % (kCols / 8);
    if (row0 + r >= half_rows || h * half_rows + row0 + r >= it.n_rows) continue;
    const int in_prob = it.row0 + h * half_rows + row0 + r, tok = P.by_group(in_prob);
    const RowWriter<D> out(P, it.shared, it.tok0 + tok, it.head * P.group + in_prob - tok * P.group,
                           true, top_s[r], sum_s[r]);
    float y[8];
    *reinterpret_cast<float4*>(y) = rows[r][2 * k];
    *reinterpret_cast<float4*>(y + 4) = rows[r][2 * k + 1];
    out.write8(z * kCols + 8 * k, y);
  }
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams P) {
  __shared__ float2 fac[kDecodeScheduleCtas][32];  // maxima and sums
  __shared__ float4 rows[32][D / 8 + 1];
  __shared__ float top_s[32], sum_s[32];
  __shared__ int before[256], warp_sum_s[8];
  pdl_wait();
  pdl_launch_dependents();
  // pieces of the item that begins in CTA `tid`: 32-row pieces of each half in use
  const int tid = threadIdx.x, lane = tid & 31, half_rows = P.rows / 2;
  auto blocks_of = [&](int rows_left) {
    return rows_left <= 0 ? 0 : (min(rows_left, half_rows) + 31) / 32;
  };
  int own = 0;
  if (tid < kDecodeScheduleCtas) {
    const SplitItem it = P.split[tid];
    if (it.parts > 1) own = 2 * (blocks_of(it.n_rows) + blocks_of(it.n_rows - half_rows));
  }
  const int incl = warp_scan(own);
  if (lane == 31) warp_sum_s[tid >> 5] = incl;
  __syncthreads();
  int base = 0, total = 0;
  for (int w = 0; w < 8; ++w) {
    if (w < tid >> 5) base += warp_sum_s[w];
    total += warp_sum_s[w];
  }
  before[tid] = base + incl - own;
  __syncthreads();
  for (int piece = blockIdx.x; piece < total; piece += kJoinBlocks) {
    int lo = 0, hi = 256;  // before[lo] <= piece < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= piece) lo = mid; else hi = mid;
    }
    const SplitItem it = P.split[lo];
    const int x = (piece - before[lo]) / 2, first = blocks_of(it.n_rows);
    const int h = x >= first ? 1 : 0;
    join_piece<D>(P, it, lo, h, (x - h * first) * 32, (piece - before[lo]) & 1, fac, rows, top_s,
                  sum_s);
  }
}

template <int D>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                   const AttnParams& P, cudaStream_t st, const DeviceInfo& dev) {
  using La = Lay<D>;
  constexpr size_t smem = 1024 + La::oMisc + sizeof(Misc<La::kSlots>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  if (smem > dev.max_smem_optin) return cudaErrorInvalidConfiguration;
  auto kern = attn_prefill_kernel<D>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kDecodeScheduleCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kern, tm_q, tm_k, tm_v, P)) != cudaSuccess || !P.join_after)
    return e;
  return launch_attn_join(P, st);
}

}  // namespace

cudaError_t launch_attn_join(const AttnParams& P, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kJoinBlocks);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return P.kv.head_dim == 64 ? cudaLaunchKernelEx(&cfg, attn_join_kernel<64>, P)
                             : cudaLaunchKernelEx(&cfg, attn_join_kernel<128>, P);
}

cudaError_t launch_attn_prefill(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                const CUtensorMap& tm_v, const AttnParams& P, cudaStream_t st,
                                const DeviceInfo& dev) {
  return P.kv.head_dim == 64 ? launch<64>(tm_q, tm_k, tm_v, P, st, dev)
                             : launch<128>(tm_q, tm_k, tm_v, P, st, dev);
}

}  // namespace lora
