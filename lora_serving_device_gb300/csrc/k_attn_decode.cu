// Attention over the paged cache for few rows per key head: single tokens,
// and short runs of them (lora_attn_paged and both phases of
// lora_attn_prefix).
//
// Mathematics, per item (up to A rows of one key head) and key tile of 128 keys:
//   S^T = K Q^T                     [128 keys, A]    tcgen05, M = the keys
//   P   = 2^(S c - m)               c = scale log2(e), m the reference maximum
//   l  += column sums of P
//   O^T += V^T [P_hi | P_lo]        [D, 2 A]         tcgen05, M = head_dim
// m is a row's maximum when it was last moved; it is moved (and l, O scaled)
// only when a score exceeds it by more than 8 in log2 units, so P stays
// below 2^8 and the usual tile costs no reduction over the keys at all, only
// a vote.  P enters as a pair of bf16 (hi and the rest, in columns of their
// own), so its product with V is exact to ~2^-16; sums and O are fp32.
//
// Bound by reading the cache: 4 D bytes a key and key head.  A tile's K and V
// are brought in by TMA, one box per page and tensor, through a ring that takes
// most of the shared memory; what the tensor cores and a softmax warpgroup
// spend on a tile is a fraction of the time its bytes need.  The keys
// stand in M, where 128 is the MMA's natural size, and the few rows in N, where
// 16 is possible: padding costs nothing that is scarce.
//
// Measured (HBM's measured rate is 6.69 TB/s): 64 tokens on 500 - 8000, 32 / 8
// heads of 128: 166 us, 6.6 TB/s; 3 tokens on 90000 - 131000: 218 us, 6.7 TB/s;
// 96 tokens on 200 - 16000 with a window of 4096, 64 / 8 heads of 64: 118 us,
// 6.2 TB/s.  One token on 500: 8.5 us, of which the share takes 2.5, the first
// page ids and tiles 2.5 and the rest is the chain of four tiles.
//
// Warps: 0 = schedule and TMA, 1 = MMA issue, 2-5 and 6-9 = softmax and epilogue.
// Every wait is bounded; on timeout the kernel raises LORA_DEVERR_TIMEOUT.
#include <cudaTypedefs.h>

#include "attn.cuh"
#include "attn_tile.cuh"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kRing = 4;      // segments that the producer may run ahead

// A rows of a row tile: 4, 8 or 16.  N is their number in Q K^T and kPV the
// columns of P and O (A for the high halves from 0, A for the rest from kPV /
// 2); the MMA wants at least 16.  W softmax warpgroups take the segments in
// turn, each with its own Q, P and O, so that one's first scores and last
// results do not keep the next segment's tiles waiting (96 windowed tokens on
// up to 16000, 64 values a head: 162 -> 131 us).
template <int D, int A>
struct Lay {
  static constexpr int W = 2;
  static constexpr int kThreads = 64 + 128 * W;
  static constexpr int N = 16;
  static constexpr int kPV = A < 16 ? 16 : 2 * A;
  static constexpr uint32_t kTile = kKeys * D * 2;  // K or V of a tile
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr uint32_t kQ = N * D * 2;
  static constexpr uint32_t kP = kPV * kKeys * 2;
  static constexpr int kPBufs = A <= 8 ? 2 : 1;
  static constexpr int kSBufs = 2;
  static constexpr int kStages = 196608u / kStage;
  static constexpr uint32_t oQ = kStages * kStage;
  static constexpr uint32_t oP = oQ + W * kQ;
  static constexpr uint32_t oMisc = oP + W * kPBufs * kP;
};

template <int D, int A>
struct Misc {
  using La = Lay<D, A>;
  static constexpr int W = La::W, kStages = La::kStages;
  Segment ring[kRing];
  // Of a row: the four warps' maxima (of a tile) and sums (of a segment).  They
  // are apart because no barrier of the warpgroup lies between the last tile's
  // maxima and the sums: one warp may add up while another still reads maxima.
  float4 red_max[W][A], red_sum[W][A];
  float m[W][A];
  int row_hi[W][A], row_lo[W][A];
  uint64_t full_k[kStages], full_v[kStages], empty[kStages];
  uint64_t s_full[W][La::kSBufs], s_empty[W][La::kSBufs];
  uint64_t p_full[W][La::kPBufs], p_done[W][La::kPBufs];
  uint64_t q_full[W], o_empty[W];
  uint64_t seg_full[kRing], seg_empty[kRing];
  uint32_t tmem;
  int abort;
  int last[W];
};

template <int D, int A>
__global__ void __launch_bounds__(Lay<D, A>::kThreads, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const AttnParams P) {
  using La = Lay<D, A>;
  constexpr int N = La::N, kPV = La::kPV;
  constexpr int W = La::W, kStages = La::kStages, PB = La::kPBufs, SB = La::kSBufs;
  using Mi = Misc<D, A>;
  constexpr uint32_t kUsed = W * (SB * N + kPV);  // S, then O
  constexpr uint32_t kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : 256;
  static_assert(kUsed <= 256, "tensor memory");
  constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(kKeys, N, false, false);
  constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(D, kPV, true, false);
  constexpr uint32_t kGroupBytes = (D / 64) * 1024;  // eight keys

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Mi& M = *reinterpret_cast<Mi*>(smem + La::oMisc);
  volatile int* abort_f = &M.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&M.full_k[i], 1);
      ptx::mbar_init(&M.full_v[i], 1);
      ptx::mbar_init(&M.empty[i], 1);
    }
    for (int w = 0; w < W; ++w) {
      for (int i = 0; i < SB; ++i) {
        ptx::mbar_init(&M.s_full[w][i], 1);
        ptx::mbar_init(&M.s_empty[w][i], 4);
      }
      for (int i = 0; i < PB; ++i) {
        ptx::mbar_init(&M.p_full[w][i], 4);
        ptx::mbar_init(&M.p_done[w][i], 1);
      }
      ptx::mbar_init(&M.q_full[w], 4);
      ptx::mbar_init(&M.o_empty[w], 4);
    }
    for (int i = 0; i < kRing; ++i) {
      ptx::mbar_init(&M.seg_full[i], 1);
      ptx::mbar_init(&M.seg_empty[i], 5);
    }
    M.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&M.tmem, kCols);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  // (the next grid may not start early: its launch slows this one's last CTAs,
  // which join parts, by more than its prologue takes)
  // After a prefix phase the grid before is this call's own, and what this one
  // reads until its first results is older: that grid has waited for it.  The
  // kernel that joins the prefix' parts lets this one start early, so schedule and
  // first tiles come in beside it (prefix of 8K, 64 tokens: 47.3 us, waiting
  // first 48.6; of 20000, 8 tokens: 40.4, 43.9).
  const bool late = P.n_groups > 0 && !P.groups_phase;
  if (!late) pdl_wait();
  // the tiles' memory holds the problems' sizes until the first load
  size_problems(P, reinterpret_cast<ProblemSize*>(smem));
  ptx::fence_proxy_async_smem();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = M.tmem;
  const uint32_t tmem_o = tmem + W * SB * N;  // after the buffers of S

  if (warp == 0) {
    // ---------------- schedule and TMA ----------------------------------
    Walker walk;
    walk.start(P, reinterpret_cast<ProblemSize*>(smem));
    ptx::fence_proxy_async_smem();
    __syncwarp();
    TileLoader<D> load(P);
    int tile = 0, ends = 0;
    bool ok = true;
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
      if (g.n == 0) {
        if (++ends == W) break;  // each warpgroup finds its own end
        continue;
      }
      load.begin(P, g);
      for (int i = 0; i < g.n; ++i, ++tile) {
        const int at = load.at(P, g, i);
        const uint32_t bytes = load.bytes(at);
        const int st = tile % kStages;
        if (tile >= kStages) ok = wait_all(&M.empty[st], ((tile / kStages) & 1) ^ 1, abort_f);
        if (!ok) break;
        uint8_t* K = smem + st * La::kStage;
        load.load(&tm_k, &M.full_k[st], K, at, bytes);
        load.load(&tm_v, &M.full_v[st], K + La::kTile, at, bytes);
      }
    }
    if (!ok) {
      // gave up: what is on its way into shared memory has to land first
      int none = 0;
      for (int k = tile > kStages ? tile - kStages : 0; k < tile; ++k) {
        ptx::mbar_wait_bounded(&M.full_k[k % kStages], (k / kStages) & 1, &none, kAttnWaitNs / 8);
        ptx::mbar_wait_bounded(&M.full_v[k % kStages], (k / kStages) & 1, &none, kAttnWaitNs / 8);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issue ------------------------------------------
    // One thread with two cursors over the same tiles: O += of tile pv as soon
    // as its P is there, S of tile qk as soon as its K is there and one of its
    // warpgroup's buffers is free.
    if (elect_one()) {
      const uint32_t stages = desc_lo(ptx::smem_u32(smem), 0);
      const uint32_t qa = desc_lo(ptx::smem_u32(smem + La::oQ), 16);
      const uint32_t pa = desc_lo(ptx::smem_u32(smem + La::oP), 16);
      uint32_t qk = 0, pv = 0;  // tiles issued
      uint32_t qs = 0, ps = 0;  // their segments
      int q_left = -1, p_left = 0;  // tiles to go in them; -1: header not read
      uint32_t s0 = 0, s1 = 0, p0 = 0, p1 = 0;  // uses of each warpgroup's S and P
      bool q_first = true, p_first = true;
      Patience wait;
      for (;;) {
        if (q_left < 0) {
          if (ptx::mbar_test_wait(&M.seg_full[qs % kRing], (qs / kRing) & 1)) {
            q_left = M.ring[qs % kRing].n;
            q_first = true;
            wait.reset();
          }
        } else if (q_left == 0 && pv == qk) {
          break;  // the end of the share
        }
        if (pv < qk) {
          if (p_left == 0) {
            p_left = M.ring[ps % kRing].n;
            p_first = true;
          }
          const uint32_t w = ps % W, use = w ? p1 : p0;
          if (ptx::mbar_test_wait(&M.p_full[w][use % PB], (use / PB) & 1) &&
              ptx::mbar_test_wait(&M.full_v[pv % kStages], (pv / kStages) & 1) &&
              (!p_first || ps < W || ptx::mbar_test_wait(&M.o_empty[w], (ps / W - 1) & 1))) {
            ptx::tc_fence_after();
            const uint32_t st = pv % kStages;
            const uint32_t va = stages + (st * La::kStage + La::kTile) / 16 + ((1024u / 16) << 16);
            const uint32_t pb = pa + (w * PB + use % PB) * (La::kP / 16);
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ++ks)
              mma_ss(tmem_o + w * kPV, va + ks * 2 * kGroupBytes / 16, desc_hi(kGroupBytes),
                     pb + ((ks / 4) * (kPV * 128) + (ks % 4) * 32) / 16, desc_hi(1024), kIdescPV,
                     ks > 0 || !p_first ? 1u : 0u);
            ptx::mma_commit(&M.empty[st]);
            ptx::mma_commit(&M.p_done[w][use % PB]);
            if (w) ++p1; else ++p0;
            ++pv;
            p_first = false;
            if (--p_left == 0) {
              ptx::mbar_arrive(&M.seg_empty[ps % kRing]);
              ++ps;
            }
            wait.reset();
            continue;
          }
        }
        const uint32_t v = qs % W, s_use = v ? s1 : s0;
        if (q_left > 0 &&
            ptx::mbar_test_wait(&M.full_k[qk % kStages], (qk / kStages) & 1) &&
            (s_use < SB || ptx::mbar_test_wait(&M.s_empty[v][s_use % SB], ((s_use / SB) & 1) ^ 1)) &&
            (!q_first || ptx::mbar_test_wait(&M.q_full[v], (qs / W) & 1))) {
          ptx::tc_fence_after();
          const uint32_t ka = stages + (qk % kStages) * (La::kStage / 16) + (1u << 16);
          const uint32_t qd = qa + v * (La::kQ / 16);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ss(tmem + (v * SB + s_use % SB) * N, ka + ((ks / 4) * 1024 + (ks % 4) * 32) / 16,
                   desc_hi(kGroupBytes), qd + ((ks / 4) * (N * 128) + (ks % 4) * 32) / 16,
                   desc_hi(1024), kIdescQK, ks > 0 ? 1u : 0u);
          ptx::mma_commit(&M.s_full[v][s_use % SB]);
          if (v) ++s1; else ++s0;
          ++qk;
          q_first = false;
          if (--q_left == 0) {
            ++qs;
            q_left = -1;
          }
          wait.reset();
          continue;
        }
        if (wait.out(abort_f)) break;
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax and epilogue --------------------------------
    const int w = warp & 3;                 // TMEM lanes 32w .. 32w + 31
    const int j = w * 32 + lane;            // this thread's key in a tile
    const int wg = (warp - 2) / 4;          // warpgroup
    const int st_tid = tid - 64 - wg * 128;
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    const bool has_d = D == 128 || lane < 16;   // M = 64 fills 16 lanes of each warp
    const int d = D == 128 ? j : w * 16 + lane;  // this thread's column of O
    const float c = P.scale_log2;
    const int kBar = 1 + wg;
    float4 *const red_max = M.red_max[wg], *const red_sum = M.red_sum[wg];
    uint8_t* const Pbase = smem + La::oP + wg * PB * La::kP;
    const uint32_t tm_o = tmem_o + wg * kPV + lanes;
    uint64_t* const p_full = M.p_full[wg];
    uint64_t* const p_done = M.p_done[wg];

    // Q of a segment into shared memory, rows past the last as zeros
    auto load_q = [&](const Segment& g) {
      uint8_t* Q = smem + La::oQ + wg * La::kQ;
#pragma unroll
      for (int i = st_tid; i < N * (D / 8); i += 128) {
        const int n = i / (D / 8), ch = i % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (n < g.t.n_rows) {
          const int r = g.t.row0 + n, tok = P.by_group(r);
          v = *reinterpret_cast<const uint4*>(
              P.q + (g.tok0 + tok) * P.q_stride +
              (g.head * P.group + r - tok * P.group) * D + ch * 8);
        }
        *reinterpret_cast<uint4*>(Q + (ch / 8) * (N * 128) + n * 128 +
                                  (((ch % 8) ^ (n & 7)) << 4)) = v;
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&M.q_full[wg]);
    };

    // The four warps meet at barriers, so none leaves on its own: after a
    // wait that gave up they run on (every later wait returns at once) to
    // the vote at the next segment.
    uint32_t tile = 0;  // tiles of this warpgroup so far
    for (int sg = wg;; sg += W) {
      wait_quiet(&M.seg_full[sg % kRing], (sg / kRing) & 1, abort_f);
      if (named_any(kBar, 128, *abort_f != 0)) break;
      const Segment g = M.ring[sg % kRing];
      if (g.n == 0) break;
      load_q(g);  // (the MMAs that read the last one's are done: so are its scores)
      // limits of the rows (rows past the last copy row 0's)
      for (int n = st_tid; n < A; n += 128) {
        const int pos = g.base + P.by_group(g.t.row0 + (n < g.t.n_rows ? n : 0));
        M.row_hi[wg][n] = P.groups_phase ? g.t.vis_hi : min(pos, g.t.vis_hi);
        M.row_lo[wg][n] = P.groups_phase ? 0 : max(window_first(P, pos), g.k_lo);
      }
      named_bar(kBar, 128);
      int min_hi = M.row_hi[wg][lane % A], max_lo = M.row_lo[wg][lane % A];
      min_hi = __reduce_min_sync(0xffffffffu, min_hi);
      max_lo = __reduce_max_sync(0xffffffffu, max_lo);
      // of each row: minus the reference maximum (log2 units; +inf: none yet)
      // and the sum over this thread's keys
      float neg[A], l[A];
#pragma unroll
      for (int n = 0; n < A; ++n) {
        neg[n] = INFINITY;
        l[n] = 0.f;
      }

#pragma unroll 1
      for (int i = 0; i < g.n; ++i, ++tile) {
        const int v0 = (g.first + i) * kKeys, v = v0 + j;  // places
        const int key0 = window_key(g.t, v0), key = key0 + j;
        const uint32_t in_cta = g.tile0 + i;
        wait_quiet(&M.s_full[wg][tile % SB], (tile / SB) & 1, abort_f);
        __syncwarp();
        ptx::tc_fence_after();
        float s[N];
#pragma unroll
        for (int n = 0; n < N; n += 16)
          ptx::tmem_ld16(tmem + lanes + (wg * SB + tile % SB) * N + n,
                         *reinterpret_cast<uint32_t(*)[16]>(s + n));
        ptx::tmem_ld_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&M.s_empty[wg][tile % SB]);
        if (key0 < max_lo || key0 + kKeys - 1 > min_hi) {
#pragma unroll
          for (int n = 0; n < A; ++n)
            s[n] = ((key <= M.row_hi[wg][n]) & (key >= M.row_lo[wg][n])) |
                           ((v < g.t.n_sink) & (v <= M.row_hi[wg][n]))
                       ? s[n]
                       : -INFINITY;
        }
        // does a score exceed its reference maximum by more than 8?
        bool up = false;
#pragma unroll
        for (int n = 0; n < A; ++n) up |= fmaf(s[n], c, neg[n]) > 8.f;
        if (named_any(kBar, 128, up)) {
#pragma unroll
          for (int n = 0; n < A; ++n) {
            const float mx = warp_max(s[n]);
            if (lane == 0) reinterpret_cast<float*>(&red_max[n])[w] = mx;
          }
          named_bar(kBar, 128);
          float fac[A];
#pragma unroll
          for (int n = 0; n < A; ++n) {
            const float4 r = red_max[n];
            const float mx = fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w)) * c;
            const float now = fminf(neg[n], -mx);
            fac[n] = neg[n] == INFINITY ? 0.f : exp2_fast(now - neg[n]);
            neg[n] = now;
            l[n] *= fac[n];
          }
          if (i > 0) {
            wait_quiet(&p_done[(tile - 1) % PB], ((tile - 1) / PB) & 1, abort_f);
            __syncwarp();
            ptx::tc_fence_after();
#pragma unroll
            for (int n = 0; n < kPV; n += 16) {
              uint32_t o[16];
              ptx::tmem_ld16(tm_o + n, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x)
                o[x] = __float_as_uint(__uint_as_float(o[x]) * fac[(n + x) % (kPV / 2) % A]);
              ptx::tmem_st16(tm_o + n, o);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
          }
        }
        if (tile_has_unseen(g.t, v0)) {
          wait_quiet(&M.full_v[in_cta % kStages], (in_cta / kStages) & 1, abort_f);
          zero_unseen_value<D>(g.t, v0, j, smem + (in_cta % kStages) * La::kStage + La::kTile);
        }
        // P's buffer is free once the product that read it is done
        if (tile >= PB) wait_quiet(&p_done[tile % PB], ((tile / PB) & 1) ^ 1, abort_f);
        uint8_t* Pb = Pbase + (tile % PB) * La::kP + (j / 64) * (kPV * 128) + (j % 8) * 2;
        const int ch = (j % 64) / 8;
#pragma unroll
        for (int n = 0; n < A; ++n) {
          const float p = exp2_fast(fmaf(s[n], c, neg[n] == INFINITY ? 0.f : neg[n]));
          l[n] += p;
          const bf16 hi = __float2bfloat16_rn(p);
          const bf16 lo = __float2bfloat16_rn(p - __bfloat162float(hi));
          *reinterpret_cast<bf16*>(Pb + n * 128 + ((ch ^ (n & 7)) << 4)) = hi;
          *reinterpret_cast<bf16*>(Pb + (kPV / 2 + n) * 128 + ((ch ^ (n & 7)) << 4)) = lo;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&p_full[tile % PB]);
      }

      // ---- the item, or this CTA's part of it, is done: O by way of P's
      // buffer to threads that hold eight values of a row each
#pragma unroll
      for (int n = 0; n < A; ++n) {
        const float x = warp_sum(l[n]);
        if (lane == 0) reinterpret_cast<float*>(&red_sum[n])[w] = x;
        if (st_tid == 0) M.m[wg][n] = -neg[n];
      }
      wait_quiet(&p_done[(tile - 1) % PB], ((tile - 1) / PB) & 1, abort_f);
      __syncwarp();
      ptx::tc_fence_after();
      float* stage = reinterpret_cast<float*>(Pbase);
#pragma unroll
      for (int n0 = 0; n0 < A; n0 += 16) {
        uint32_t oh[16], ol[16];
        ptx::tmem_ld16(tm_o + n0, oh);
        if (A >= 16) ptx::tmem_ld16(tm_o + kPV / 2 + n0, ol);
        ptx::tmem_ld_wait();
        if (has_d) {
#pragma unroll
          for (int x = 0; x < (A < 16 ? A : 16); ++x)
            stage[(n0 + x) * D + d] = __uint_as_float(oh[x]) +
                                      __uint_as_float(A >= 16 ? ol[x] : oh[x + 8]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&M.o_empty[wg]);
        ptx::mbar_arrive(&M.seg_empty[sg % kRing]);
      }
      named_bar(kBar, 128);
      if (late) pdl_wait();  // the prior parts are read, and the parts' memory is free
      float2* ml = reinterpret_cast<float2*>(P.part_ml);
      const int vectors = g.t.n_rows * (D / 8);
      bool write = true;
      if (g.parts > 1) {
        const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + g.slot;
#pragma unroll 1
        for (int x = st_tid; x < vectors; x += 128) {
          const int n = x / (D / 8), k = x % (D / 8) * 8;
          store8(P.part + (slot * A + n) * D + k,
                 *reinterpret_cast<const float(*)[8]>(stage + n * D + k));
          const float4 r = red_sum[n];
          if (k == 0) ml[slot * A + n] = make_float2(M.m[wg][n], r.x + r.y + r.z + r.w);
        }
        write = last_to_arrive(P, g, 0, st_tid == 0, &M.last[wg], kBar, 128);
      }
#pragma unroll 1
      for (int x = write ? st_tid : vectors; x < vectors; x += 128) {
        const int n = x / (D / 8), k = x % (D / 8) * 8;
        float o[8], top, sum;
        if (g.parts == 1) {
          const float4 r = red_sum[n];
          top = M.m[wg][n];
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
        const RowWriter<D> out(P, g.shared, g.tok0 + tok,
                               g.head * P.group + r - tok * P.group, true, top, sum);
        out.write8(k, o);
      }
      named_bar(kBar, 128);  // the sums and the limits are free
    }
  }

  pdl_wait();  // (a CTA without items too: this grid ends after the one before)
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kCols);
  }
  if (tid == 0 && *abort_f) flag_error(P.err, LORA_DEVERR_TIMEOUT);
}

template <int D, int A>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnParams& P,
                   cudaStream_t st, const DeviceInfo& dev) {
  using La = Lay<D, A>;
  constexpr size_t smem = 1024 + La::oMisc + sizeof(Misc<D, A>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  if (smem > dev.max_smem_optin) return cudaErrorInvalidConfiguration;
  auto kern = attn_decode_kernel<D, A>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kDecodeScheduleCtas);
  cfg.blockDim = dim3(La::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, P);
}

}  // namespace

cudaError_t launch_attn_decode(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                               const AttnParams& P, cudaStream_t st, const DeviceInfo& dev) {
  if (P.kv.head_dim == 64) {
    switch (P.rows) {
      case 4: return launch<64, 4>(tm_k, tm_v, P, st, dev);
      case 8: return launch<64, 8>(tm_k, tm_v, P, st, dev);
      default: return launch<64, 16>(tm_k, tm_v, P, st, dev);
    }
  }
  switch (P.rows) {
    case 4: return launch<128, 4>(tm_k, tm_v, P, st, dev);
    case 8: return launch<128, 8>(tm_k, tm_v, P, st, dev);
    default: return launch<128, 16>(tm_k, tm_v, P, st, dev);
  }
}

}  // namespace lora
