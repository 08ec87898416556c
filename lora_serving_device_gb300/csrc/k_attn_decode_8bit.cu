// Attention over the 8-bit paged cache for few rows per key head: single tokens,
// and short runs of them (lora_attn_paged_8bit and both phases of
// lora_attn_prefix_8bit).
//
// The codes go to the tensor cores as they lie in memory; what is not 8 bits is made
// so, exactly enough.  Per item (up to A rows of one key head) and key tile of 128:
//   S^T = K [Q_1 + Q_2]^T          [128 keys, A]    e4m3, M = the keys
//   s   = c 2^(kb + qb) S^T        kb, qb the exponents of a key's block and a row
//   P   = 2^(s - m),  l += column sums of P
//   O^T += V^T [P_1 | P_2 | P_3]   [D, 3 A]         e4m3, P 2^(vb - R) in three terms
// Q: a row divided by a power of two that puts its largest value into (224, 448] is
// the sum of two e4m3 terms, off by at most 2^-10 there.  P: a term holds four bits, and the
// next one what it leaves, 2^4 times as large, so three are exact to 2^-12 of P, or
// 2^-23 where P is small; they are columns of their own, added at the end.
// m is a row's maximum less 5 when it was last moved (as in the bf16 kernel, but moved at
// 3 log2 units above: P stays below 2^8 and its largest value above 2^5).  R is the
// largest exponent of a value block so far; O is scaled when it grows.
//
// Bound by reading the cache: 2 D bytes a key and key head.  Converting the codes
// instead (to bf16, for the other kernel's loop) would move each tile through
// registers and write it to shared memory at twice its size, 1.5 times what the shared memory
// passes in the time that the tile's bytes take; here nothing touches it on the way.
// A key's two exponents belong to the thread that owns the key, so scales cost two
// multiplications; a warp of its own looks them up, tiles ahead.
// The terms of P lie as [key][term, row]: a thread stores its key's in 16 bytes at once.
//
// Measured (HBM's measured rate is 6.69 TB/s): 64 tokens on 500 - 8000, 32 / 8 heads of 128,
// pages of 16: 90 us, 6.1 TB/s; 152 on 4000 186 us, 6.7 TB/s; 3 tokens on 90000 - 131000: 117 us,
// 6.3 TB/s; one token on 500 9.2 us; 96 tokens with a window of 4096, 64 / 8 heads of 64, 102 us, 3.6 TB/s.  With
// 9 to 16 rows of a key head one buffer of P is all that fits, and 36 (128 values a head) or 44 bytes
// spill: 64 tokens on 8K with 32 / 2 heads of 128 42 us, 3.6 TB/s, with 64 / 4 of 64 58 us.  A batch of few items a CTA pays its first page ids,
// tiles and results: 19 tokens on 8000, one item a CTA, 52 us, 6.0 TB/s.
//
// Warps: 0 = schedule and TMA of K, 1 = MMA issue, 2-5 and 6-9 = softmax and epilogue, 10 =
// scales, 11 = TMA of V.  Every wait is bounded; on timeout the kernel raises LORA_DEVERR_TIMEOUT.
#include <cudaTypedefs.h>

#include "attn.cuh"
#include "attn_tile.cuh"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kRing = 4;      // segments that the producer may run ahead
constexpr float kTop = 5.f;   // log2 of a row's largest weight when its reference is set
constexpr float kTerm = 16.f; // a term of P against the one before

// A rows of a row tile: 4, 8 or 16.  N is their number in Q K^T and kPV the columns of P
// and O (three terms of A rows, in whole planes of 16).  W softmax warpgroups take the
// segments in turn, each with its own Q, P and O.
template <int D, int A>
struct Lay {
  static constexpr int W = 2;
  static constexpr int kThreads = 128 + 128 * W;
  static constexpr int N = 16;
  static constexpr int kPV = (3 * A + 15) / 16 * 16;
  static constexpr uint32_t kTile = kKeys * D;  // K or V of a tile
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr uint32_t kQ = 2 * N * D;
  static constexpr uint32_t kPlane = kKeys * 16;  // 16 columns of P
  static constexpr uint32_t kP = kPV * kKeys;
  static constexpr int kPBufs = A <= 8 ? 2 : 1;
  static constexpr uint32_t kStaging = A * D * 4;  // results on their way out, in P's place
  static constexpr uint32_t kPAll = kPBufs * kP > kStaging ? kPBufs * kP : kStaging;
  static constexpr int kSBufs = 2;
  static constexpr int kStages = 196608u / kStage;
  // A warpgroup waits for the scales of its own segments only, by one bit of a barrier's phase: when it
  // comes for a segment's first batch, the one before it in the ring's place has to be there.  The
  // header that it comes by follows the last key tile of the other's segment, so kStages tiles of that may
  // be without scales: their batches, of two tiles at least but for the last, have to be fewer than the ring's.
  static constexpr int kScaleBatches = D == 128 ? 4 : 8;
  static_assert(1 + (kStages - 1) / 2 < kScaleBatches, "a batch of scales two phases behind");
  static constexpr uint32_t oQ = kStages * kStage;
  static constexpr uint32_t oP = oQ + W * kQ;
  static constexpr uint32_t oMisc = oP + W * kPAll;
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
  float q_scale[W][La::N];
  ScaleRing<La::kScaleBatches> scales;
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

// After a wait that gave up: what is on its way into shared memory has to land first.
__device__ __forceinline__ void drain(uint64_t* full, int stages, int tiles) {
  int none = 0;
  for (int k = tiles > stages ? tiles - stages : 0; k < tiles; ++k)
    ptx::mbar_wait_bounded(&full[k % stages], (k / stages) & 1, &none, kAttnWaitNs / 8);
}

template <int D, int A>
__global__ void __launch_bounds__(Lay<D, A>::kThreads, 1)
    attn_decode_8bit_kernel(const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const AttnParams P) {
  using La = Lay<D, A>;
  constexpr int N = La::N, kPV = La::kPV;
  constexpr int W = La::W, kStages = La::kStages, PB = La::kPBufs, SB = La::kSBufs;
  using Mi = Misc<D, A>;
  constexpr uint32_t kUsed = W * (SB * N + kPV);  // S, then O
  constexpr uint32_t kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : 256;
  static_assert(kUsed <= 256, "tensor memory");
  constexpr uint32_t kIdescQK = ptx::idesc_e4m3_f32(kKeys, N, false, false);
  constexpr uint32_t kIdescPV = ptx::idesc_e4m3_f32(D, kPV, true, true);
  constexpr uint32_t kGroupBytes = 8 * D;  // eight keys

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
      ptx::mbar_init(&M.seg_empty[i], 7);
    }
    init_scales(M.scales, 4);
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
  // (the tokens' phase after a prefix phase begins before the grid before it has ended, and
  // waits for it before its first result, as in the bf16 kernel)
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
    TileLoader<D, 1> load(P);
    int tile = 0, ends = 0, batches = 0;
    bool ok = true;
    for (int sg = 0; ok; ++sg) {
      Segment g = walk.next(P);
      g.batch0 = batches;
      batches += (g.n + P.scale_tiles - 1) >> (P.scale_tiles == 2 ? 1 : 2);
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
        load.load(&tm_k, &M.full_k[st], smem + st * La::kStage, at, bytes);
      }
    }
    if (!ok) drain(M.full_k, kStages, tile);
  } else if (warp == 1) {
    // ---------------- MMA issue ------------------------------------------
    // One thread with two cursors over the same tiles: O += of tile pv as soon
    // as its P is there, S of tile qk as soon as its K is there and one of its
    // warpgroup's buffers is free.
    if (elect_one()) {
      const uint32_t stages = desc_lo(ptx::smem_u32(smem), 0);
      const uint32_t qa = desc_lo(ptx::smem_u32(smem + La::oQ), 16);
      // P: eight keys of a plane are 128 bytes, planes are kPlane apart
      const uint32_t pa = desc_lo(ptx::smem_u32(smem + La::oP), 128);
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
            const uint32_t pb = pa + (w * La::kPAll + use % PB * La::kP) / 16;
#pragma unroll
            for (int ks = 0; ks < kKeys / 32; ++ks)
              mma_ss_8bit(tmem_o + w * kPV, va + ks * 4 * kGroupBytes / 16,
                          desc_hi_span(kGroupBytes, D), pb + ks * 4 * 128 / 16,
                          desc_hi_span(La::kPlane, 0), kIdescPV, ks > 0 || !p_first ? 1u : 0u);
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
          // Q's terms, of 128 bytes a row: one plane each, or halves of one with D = 64
#pragma unroll
          for (int ks = 0; ks < 2 * D / 32; ++ks)
            mma_ss_8bit(tmem + (v * SB + s_use % SB) * N, ka + ks % (D / 32) * 2,
                        desc_hi_span(kGroupBytes, D),
                        qd + ((ks / 4) * (N * 128) + (ks % 4) * 32) / 16, desc_hi(1024), kIdescQK,
                        ks > 0 ? 1u : 0u);
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
  } else if (warp == 10) {
    // ---------------- scales ----------------------------------------------
    run_scales(P, M.scales, M.ring, kRing, M.seg_full, M.seg_empty, abort_f);
  } else if (warp == 11) {
    // ---------------- TMA of V ---------------------------------------------
    // A warp of its own: a box takes the warp that issues it ~40 ns, and pages of 16 tokens
    // make 16 boxes a tile (64 tokens on 8K: one warp for K and V 109 us).
    TileLoader<D, 1> load(P);
    int tile = 0;
    bool ok = true;
    for (int sg = 0; ok; ++sg) {
      ok = wait_all(&M.seg_full[sg % kRing], (sg / kRing) & 1, abort_f);
      if (!ok) break;
      const Segment g = M.ring[sg % kRing];
      if (g.n == 0) break;
      load.begin(P, g);
      for (int i = 0; i < g.n; ++i, ++tile) {
        const int at = load.at(P, g, i);
        const uint32_t bytes = load.bytes(at);
        const int st = tile % kStages;
        if (tile >= kStages) ok = wait_all(&M.empty[st], ((tile / kStages) & 1) ^ 1, abort_f);
        if (!ok) break;
        load.load(&tm_v, &M.full_v[st], smem + st * La::kStage + La::kTile, at, bytes);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&M.seg_empty[sg % kRing]);
    }
    if (!ok) drain(M.full_v, kStages, tile);
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
    uint8_t* const Pbase = smem + La::oP + wg * La::kPAll;
    const int my_block = j / min(P.kv.page_size, kScaleBlock);
    const uint32_t tm_o = tmem_o + wg * kPV + lanes;
    uint64_t* const p_full = M.p_full[wg];
    uint64_t* const p_done = M.p_done[wg];

    // Q of a segment into shared memory as two terms, rows past the last as zeros: eight
    // threads to a row
    auto load_q = [&](const Segment& g) {
      constexpr int kPer = D / 8;  // values of a thread
      uint8_t* Q = smem + La::oQ + wg * La::kQ;
      const int n = st_tid / 8, i = st_tid % 8;
      float x[kPer];
      float top = 0.f;
#pragma unroll
      for (int y = 0; y < kPer; ++y) x[y] = 0.f;
      if (n < g.t.n_rows) {
        const int r = g.t.row0 + n, tok = P.by_group(r);
        const bf16* from = P.q + (g.tok0 + tok) * P.q_stride +
                           (g.head * P.group + r - tok * P.group) * D + i * kPer;
#pragma unroll
        for (int y = 0; y < kPer; y += 8) load8(from + y, *reinterpret_cast<float(*)[8]>(x + y));
#pragma unroll
        for (int y = 0; y < kPer; ++y) top = fmaxf(top, fabsf(x[y]));
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int byte = min(scale_byte(top), 253);
      const float inv = scale_of(254 - byte);
      uint32_t t1[kPer / 4], t2[kPer / 4];
#pragma unroll
      for (int y = 0; y < kPer / 4; ++y) {
        float* z = x + 4 * y;
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] *= inv;
        t1[y] = pack4_e4m3(z[0], z[1], z[2], z[3]);
        const float2 lo = unpack2_e4m3(t1[y]), hi = unpack2_e4m3(t1[y] >> 16);
        t2[y] = pack4_e4m3(z[0] - lo.x, z[1] - lo.y, z[2] - hi.x, z[3] - hi.y);
      }
      if (D == 128) {
        uint8_t* to = Q + n * 128 + ((i ^ (n & 7)) << 4);
        *reinterpret_cast<uint4*>(to) = make_uint4(t1[0], t1[1], t1[kPer / 4 - 2], t1[kPer / 4 - 1]);
        *reinterpret_cast<uint4*>(to + N * 128) =
            make_uint4(t2[0], t2[1], t2[kPer / 4 - 2], t2[kPer / 4 - 1]);
      } else {
        uint8_t* row = Q + n * 128 + (i & 1) * 8;
        *reinterpret_cast<uint2*>(row + ((i / 2 ^ (n & 7)) << 4)) = make_uint2(t1[0], t1[1]);
        *reinterpret_cast<uint2*>(row + (((4 + i / 2) ^ (n & 7)) << 4)) = make_uint2(t2[0], t2[1]);
      }
      if (i == 0) M.q_scale[wg][n] = scale_of(byte);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&M.q_full[wg]);
    };

    // The four warps meet at barriers, so none leaves on its own: after a
    // wait that gave up they run on (every later wait returns at once) to
    // the vote at the next segment.
    uint32_t tile = 0;  // tiles of this warpgroup so far
    const ScaleReader scales(P);
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
      // of each row: minus the reference maximum (log2 units; +inf: none yet), the sum
      // over this thread's keys, and what its scores are to be multiplied with
      float neg[A], l[A], q_scale[A];
#pragma unroll
      for (int n = 0; n < A; ++n) {
        neg[n] = INFINITY;
        l[n] = 0.f;
        q_scale[n] = M.q_scale[wg][n];
      }
      int R = 0;  // the largest exponent of a value block so far

#pragma unroll 1
      for (int i = 0; i < g.n; ++i, ++tile) {
        const int v0 = (g.first + i) * kKeys, v = v0 + j;  // places
        const int key0 = window_key(g.t, v0), key = key0 + j;
        const uint32_t in_cta = g.tile0 + i;
        const int sc = scales.of(M.scales, g, i, abort_f);
        const float kc = M.scales.k[sc][my_block] * c;
        const int vb = M.scales.v[sc][my_block], top_v = M.scales.top[sc];
        scales.done(M.scales, g, i);
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
#pragma unroll
        for (int n = 0; n < A; ++n) s[n] *= kc * q_scale[n];
        if (key0 < max_lo || key0 + kKeys - 1 > min_hi) {
#pragma unroll
          for (int n = 0; n < A; ++n)
            s[n] = ((key <= M.row_hi[wg][n]) & (key >= M.row_lo[wg][n])) |
                           ((v < g.t.n_sink) & (v <= M.row_hi[wg][n]))
                       ? s[n]
                       : -INFINITY;
        }
        // does a score exceed its reference by more than 8, or a scale R?
        bool up = top_v > R;
#pragma unroll
        for (int n = 0; n < A; ++n) up |= s[n] + neg[n] > 8.f;
        if (named_any(kBar, 128, up)) {
#pragma unroll
          for (int n = 0; n < A; ++n) {
            const float mx = warp_max(s[n]);
            if (lane == 0) reinterpret_cast<float*>(&red_max[n])[w] = mx;
          }
          named_bar(kBar, 128);
          const float fac_v = top_v - R < 127 ? scale_of(127 - (top_v - R)) : 0.f;
          R = top_v;
          float fac[A];
#pragma unroll
          for (int n = 0; n < A; ++n) {
            const float4 r = red_max[n];
            const float mx = fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w));
            const float now = fminf(neg[n], kTop - mx);
            fac[n] = neg[n] == INFINITY ? 0.f : exp2_fast(now - neg[n]);
            neg[n] = now;
            l[n] *= fac[n];
            fac[n] *= fac_v;
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
                o[x] = __float_as_uint(__uint_as_float(o[x]) * fac[(n + x) % A]);
              ptx::tmem_st16(tm_o + n, o);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
          }
        }
        if (tile_has_unseen(g.t, v0)) {
          wait_quiet(&M.full_v[in_cta % kStages], (in_cta / kStages) & 1, abort_f);
          if (!place_seen(g.t, v)) {
            uint8_t* row = smem + (in_cta % kStages) * La::kStage + La::kTile + j * D;
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
              *reinterpret_cast<uint4*>(row + ((x + j) % (D / 16)) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        // P's buffer is free once the product that read it is done
        if (tile >= PB) wait_quiet(&p_done[tile % PB], ((tile / PB) & 1) ^ 1, abort_f);
        const float fv = R - vb < 127 ? scale_of(127 - (R - vb)) : 0.f;
        uint32_t terms[kPV / 4] = {};  // [term][row] and padding
#pragma unroll
        for (int n = 0; n < A; n += 4) {
          float p[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            p[x] = exp2_fast(s[n + x] + (neg[n + x] == INFINITY ? 0.f : neg[n + x]));
            l[n + x] += p[x];
            p[x] *= fv;
          }
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            const uint32_t t = pack4_e4m3(p[0], p[1], p[2], p[3]);
            terms[(term * A + n) / 4] = t;
            const float2 lo = unpack2_e4m3(t), hi = unpack2_e4m3(t >> 16);
            p[0] = fmaf(p[0], kTerm, -kTerm * lo.x);
            p[1] = fmaf(p[1], kTerm, -kTerm * lo.y);
            p[2] = fmaf(p[2], kTerm, -kTerm * hi.x);
            p[3] = fmaf(p[3], kTerm, -kTerm * hi.y);
          }
        }
        uint8_t* Pb = Pbase + (tile % PB) * La::kP + j * 16;
#pragma unroll
        for (int n = 0; n < kPV / 16; ++n)
          *reinterpret_cast<uint4*>(Pb + n * La::kPlane) =
              make_uint4(terms[4 * n], terms[4 * n + 1], terms[4 * n + 2], terms[4 * n + 3]);
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
      float o[kPV];
#pragma unroll
      for (int n = 0; n < kPV; n += 16)
        ptx::tmem_ld16(tm_o + n, *reinterpret_cast<uint32_t(*)[16]>(o + n));
      ptx::tmem_ld_wait();
      if (has_d) {
#pragma unroll
        for (int n = 0; n < A; ++n)
          stage[n * D + d] = o[n] + (1.f / kTerm) * (o[A + n] + (1.f / kTerm) * o[2 * A + n]);
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&M.o_empty[wg]);
        ptx::mbar_arrive(&M.seg_empty[sg % kRing]);
      }
      named_bar(kBar, 128);
      if (late) pdl_wait();  // the prior parts are read, and the parts' memory is free
      finish_rows<D, A, true>(P, g, stage, M.m[wg], red_sum, st_tid, &M.last[wg], kBar,
                              scale_of(max(R, 1)));
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
  auto kern = attn_decode_8bit_kernel<D, A>;
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

cudaError_t launch_attn_decode_8bit(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
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
