// Attention over the paged cache for few rows per key head: single tokens,
// and short runs of them (lora_attn_paged and both phases of
// lora_attn_prefix).
//
// Mathematics, per item (kN rows of one key head) and key tile of 128 keys:
//   S^T = K Q^T                     [128 keys, kN]   tcgen05, M = the keys
//   P   = 2^(S c - m)               c = scale log2(e), m the reference maximum
//   l  += column sums of P
//   O^T += V^T [P_hi | P_lo]        [D, 2 kN]        tcgen05, M = head_dim
// m is a row's maximum when it was last moved; it is moved (and l, O scaled)
// only when a score exceeds it by more than 8 in log2 units, so P stays
// below 2^8 and the usual tile costs no reduction over the keys at all, only
// a vote.  P enters as a pair of bf16 (hi and the rest, in columns of their
// own), so its product with V is exact to ~2^-16; sums and O are fp32.
//
// Bound by reading the cache: 4 D bytes a key and key head.  A tile's K and V
// are brought in by TMA, one box per page and tensor, through a ring that takes
// most of the shared memory; what the tensor cores and the one softmax
// warpgroup spend on a tile is a fraction of the time its bytes need.  The keys
// stand in M, where 128 is the MMA's natural size, and the few rows in N, where
// 16 is possible: padding costs nothing that is scarce.
//
// Warps: 0 = schedule and TMA, 1 = MMA issue, 2-5 = softmax and epilogue.
// Every wait is bounded; on timeout the kernel raises LORA_DEVERR_TIMEOUT.
#include <cudaTypedefs.h>

#include "attn.cuh"
#include "attn_tile.cuh"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kThreads = 192;
constexpr int kCoarse = 512;  // entries of the schedule's prefix sums
constexpr int kRing = 4;  // segments that the producer may run ahead

template <int D, int N>
struct Lay {
  static constexpr uint32_t kTile = kKeys * D * 2;  // K or V of a tile
  static constexpr uint32_t kStage = 2 * kTile;
  static constexpr uint32_t kQ = N * D * 2;
  static constexpr uint32_t kP = 2 * N * kKeys * 2;
  static constexpr int kPBufs = N <= 16 ? 2 : 1;
  static constexpr int kStages = (N <= 32 ? 196608u : 131072u) / kStage;
  static constexpr uint32_t oQ = kStages * kStage;
  static constexpr uint32_t oP = oQ + kQ;
  static constexpr uint32_t oMisc = oP + kPBufs * kP;
};

template <int N, int kStages>
struct Misc {
  Schedule<kCoarse> sched;
  Segment ring[kRing];
  float red[4][N];       // per warp maxima or sums
  float m[N], fac[N];    // reference maxima (log2 units), rescale factors
  int row_hi[N], row_lo[N];
  uint64_t full_k[kStages], full_v[kStages], empty[kStages];
  uint64_t s_full[2], s_empty[2], p_full[2], p_done[2];
  uint64_t q_full, o_empty;
  uint64_t seg_full[kRing], seg_empty[kRing];
  uint32_t tmem;
  int abort;
  int last;
};

template <int D, int N>
__global__ void __launch_bounds__(kThreads, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const AttnParams P) {
  using La = Lay<D, N>;
  constexpr int kStages = La::kStages, PB = La::kPBufs;
  using Mi = Misc<N, kStages>;
  constexpr uint32_t kCols = 4 * N < 32 ? 32 : 4 * N;  // S twice, O's two halves
  constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(kKeys, N, false, false);
  constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(D, 2 * N, true, false);
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
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&M.s_full[i], 1);
      ptx::mbar_init(&M.s_empty[i], 4);
      ptx::mbar_init(&M.p_full[i], 4);
      ptx::mbar_init(&M.p_done[i], 1);
    }
    ptx::mbar_init(&M.q_full, 4);
    ptx::mbar_init(&M.o_empty, 4);
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
  pdl_wait();
  pdl_launch_dependents();
  build_schedule(P, M.sched);  // ends with a barrier
  ptx::tc_fence_after();
  const uint32_t tmem = M.tmem;
  const uint32_t tmem_o = tmem + 2 * N;

  if (warp == 0) {
    // ---------------- schedule and TMA ----------------------------------
    Walker<kCoarse> walk;
    walk.start(P, M.sched);
    const TileLoader<D> load(P);
    int tile = 0;
    bool ok = true;
    for (int sg = 0; ok; ++sg) {
      const Segment g = walk.next(P, M.sched);
      if (sg >= kRing)
        ok = wait_all(&M.seg_empty[sg % kRing], ((sg / kRing) & 1) ^ 1, abort_f);
      if (!ok) break;
      if (lane == 0) {
        M.ring[sg % kRing] = g;
        ptx::mbar_arrive(&M.seg_full[sg % kRing]);
      }
      __syncwarp();
      if (g.n == 0) break;
      int at = load.lookup(P, g, 0);  // page ids a tile ahead
      for (int i = 0; i < g.n; ++i, ++tile) {
        const int here = at;
        if (i + 1 < g.n) at = load.lookup(P, g, i + 1);
        const int st = tile % kStages;
        if (tile >= kStages) ok = wait_all(&M.empty[st], ((tile / kStages) & 1) ^ 1, abort_f);
        if (!ok) break;
        uint8_t* K = smem + st * La::kStage;
        load.load(&tm_k, &M.full_k[st], K, here);
        load.load(&tm_v, &M.full_v[st], K + La::kTile, here);
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
    // Two cursors over the same tiles: S of tile qk as soon as its K is
    // there, O += of tile pv as soon as its P is.  S runs at most two ahead.
    int qk = 0, pv = 0;             // tiles issued
    int qs = 0, ps = 0;             // their segments
    int qi = 0, pi = 0;             // their numbers in them
    int q_n = -1, p_n = -1;         // segment sizes, -1: not read yet
    const uint32_t qa = ptx::smem_u32(smem + La::oQ);
    Patience wait;
    while (!(q_n == 0 && pv == qk)) {
      int did = 0;
      // segment headers
      if (q_n < 0 && __all_sync(0xffffffffu, ptx::mbar_test_wait(&M.seg_full[qs % kRing],
                                                                 (qs / kRing) & 1))) {
        q_n = M.ring[qs % kRing].n;
        did = 1;
      }
      if (pv < qk && p_n < 0) {
        p_n = M.ring[ps % kRing].n;  // the other cursor has been here
        did = 1;
      }
      int go = 0;
      if (lane == 0) {
        if (pv < qk && ptx::mbar_test_wait(&M.p_full[pv % PB], (pv / PB) & 1) &&
            ptx::mbar_test_wait(&M.full_v[pv % kStages], (pv / kStages) & 1) &&
            (pi > 0 || ps == 0 || ptx::mbar_test_wait(&M.o_empty, (ps - 1) & 1)))
          go = 1;
        else if (q_n > 0 && qk - pv < 2 &&
                 ptx::mbar_test_wait(&M.full_k[qk % kStages], (qk / kStages) & 1) &&
                 (qk < 2 || ptx::mbar_test_wait(&M.s_empty[qk & 1], ((qk >> 1) & 1) ^ 1)) &&
                 (qi > 0 || ptx::mbar_test_wait(&M.q_full, qs & 1)))
          go = 2;
      }
      go = __shfl_sync(0xffffffffu, go, 0);
      if (go == 1) {
        const Segment& g = M.ring[ps % kRing];
        const int st = pv % kStages;
        uint8_t* V = smem + st * La::kStage + La::kTile;
        zero_unseen_values<D>(g.t, key_tile(g.t, g.first + pi), V);
        ptx::tc_fence_after();
        if (lane == 0) {
          const uint32_t va = ptx::smem_u32(V);
          const uint32_t pa = ptx::smem_u32(smem + La::oP + (pv % PB) * La::kP);
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks) {
            const uint64_t vd =
                ptx::sdesc_sw128(va + ks * 2 * kGroupBytes, 1024, kGroupBytes);
            const uint64_t pd = ptx::sdesc_sw128(
                pa + (ks / 4) * (2 * N * 128) + (ks % 4) * 32, 16, 1024);
            ptx::mma_bf16(tmem_o, vd, pd, kIdescPV, pi > 0 || ks > 0 ? 1u : 0u);
          }
          ptx::mma_commit(&M.empty[st]);
          ptx::mma_commit(&M.p_done[pv % PB]);
        }
        __syncwarp();
        ++pv;
        if (++pi == p_n) {
          if (lane == 0) ptx::mbar_arrive(&M.seg_empty[ps % kRing]);
          ++ps;
          pi = 0;
          p_n = -1;
        }
        did = 1;
      } else if (go == 2) {
        ptx::tc_fence_after();
        if (lane == 0) {
          const uint32_t ka = ptx::smem_u32(smem + (qk % kStages) * La::kStage);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t kd =
                ptx::sdesc_sw128(ka + (ks / 4) * 1024 + (ks % 4) * 32, 16, kGroupBytes);
            const uint64_t qd =
                ptx::sdesc_sw128(qa + (ks / 4) * (N * 128) + (ks % 4) * 32, 16, 1024);
            ptx::mma_bf16(tmem + (qk & 1) * N, kd, qd, kIdescQK, ks > 0 ? 1u : 0u);
          }
          ptx::mma_commit(&M.s_full[qk & 1]);
        }
        __syncwarp();
        ++qk;
        if (++qi == q_n) {
          ++qs;
          qi = 0;
          q_n = -1;
        }
        did = 1;
      }
      if (!__any_sync(0xffffffffu, did) && wait.out(abort_f)) break;
      if (did) wait.reset();
    }
  } else {
    // ---------------- softmax and epilogue --------------------------------
    const int w = warp & 3;                 // TMEM lanes 32w .. 32w + 31
    const int j = w * 32 + lane;            // this thread's key in a tile
    const int st_tid = tid - 64;
    const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
    const bool has_d = D == 128 || lane < 16;   // M = 64 fills 16 lanes of each warp
    const int d = D == 128 ? j : w * 16 + lane;  // this thread's column of O
    const float c = P.scale_log2;
    constexpr int kBar = 1;
    float l[N];

    // Q of a segment into shared memory, rows past the last as zeros
    auto load_q = [&](const Segment& g) {
      uint8_t* Q = smem + La::oQ;
      for (int i = st_tid; i < N * (D / 8); i += 128) {
        const int n = i / (D / 8), ch = i % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (n < g.t.n_rows) {
          const int r = g.t.row0 + n;
          v = *reinterpret_cast<const uint4*>(
              P.q + (g.tok0 + r / P.group) * P.q_stride +
              (g.head * P.group + r % P.group) * D + ch * 8);
        }
        *reinterpret_cast<uint4*>(Q + (ch / 8) * (N * 128) + n * 128 +
                                  (((ch % 8) ^ (n & 7)) << 4)) = v;
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&M.q_full);
    };
    auto seg_wait = [&](int s) {
      return wait_all(&M.seg_full[s % kRing], (s / kRing) & 1, abort_f);
    };

    // The four warps meet at barriers, so none leaves on its own: after a
    // wait that gave up they run on (every later wait returns at once) to
    // the vote at the segment's end.
    int tile = 0;  // tiles of this CTA so far
    bool ok = seg_wait(0);
    if (ok && M.ring[0].n > 0) load_q(M.ring[0]);
    for (int sg = 0; !named_any(kBar, 128, !ok); ++sg) {
      const Segment g = M.ring[sg % kRing];
      if (g.n == 0) break;
      // limits of the rows (rows past the last copy row 0's) and a first m
      for (int n = st_tid; n < N; n += 128) {
        const int pos = g.base + (g.t.row0 + (n < g.t.n_rows ? n : 0)) / P.group;
        M.row_hi[n] = P.groups_phase ? g.t.vis_hi : min(pos, g.t.vis_hi);
        M.row_lo[n] =
            P.groups_phase ? 0 : max(P.window > 0 ? max(pos - P.window + 1, 0) : 0, g.k_lo);
        M.m[n] = -INFINITY;
        M.fac[n] = 0.f;
      }
      named_bar(kBar, 128);
      int min_hi = M.row_hi[lane % N], max_lo = M.row_lo[lane % N];
      if (N > 32) {
        min_hi = min(min_hi, M.row_hi[(lane + 32) % N]);
        max_lo = max(max_lo, M.row_lo[(lane + 32) % N]);
      }
      min_hi = __reduce_min_sync(0xffffffffu, min_hi);
      max_lo = __reduce_max_sync(0xffffffffu, max_lo);
#pragma unroll
      for (int n = 0; n < N; ++n) l[n] = 0.f;

      for (int i = 0; i < g.n; ++i, ++tile) {
        const int key0 = key_tile(g.t, g.first + i) * kKeys, key = key0 + j;
        ok &= wait_all(&M.s_full[tile & 1], (tile >> 1) & 1, abort_f);
        ptx::tc_fence_after();
        float s[N];
#pragma unroll
        for (int n = 0; n < N; n += 16)
          ptx::tmem_ld16(tmem + lanes + (tile & 1) * N + n,
                         *reinterpret_cast<uint32_t(*)[16]>(s + n));
        ptx::tmem_ld_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&M.s_empty[tile & 1]);
        if (i == g.n - 1) {
          // the last S is here, so Q's buffer is free: fetch the next one's
          ok &= seg_wait(sg + 1);
          if (ok && M.ring[(sg + 1) % kRing].n > 0) load_q(M.ring[(sg + 1) % kRing]);
        }
        if (key0 < max_lo || key0 + kKeys - 1 > min_hi) {
#pragma unroll
          for (int n = 0; n < N; ++n)
            if (key > M.row_hi[n] || (key < M.row_lo[n] && key >= g.t.n_sink)) s[n] = -INFINITY;
        }
        // does a score exceed its reference maximum by more than 8?
        bool up = false;
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (n < g.t.n_rows) up |= fmaf(s[n], c, -M.m[n]) > 8.f;
        if (named_any(kBar, 128, up)) {
#pragma unroll
          for (int n = 0; n < N; ++n) {
            if (n < g.t.n_rows) {
              const float mx = warp_max(s[n]);
              if (lane == 0) M.red[w][n] = mx;
            }
          }
          named_bar(kBar, 128);
          for (int n = st_tid; n < g.t.n_rows; n += 128) {
            const float mx =
                fmaxf(fmaxf(M.red[0][n], M.red[1][n]), fmaxf(M.red[2][n], M.red[3][n])) * c;
            const float old = M.m[n], now = fmaxf(old, mx);
            M.fac[n] = old == -INFINITY ? 0.f : exp2_fast(old - now);
            M.m[n] = now;
          }
          named_bar(kBar, 128);
#pragma unroll
          for (int n = 0; n < N; ++n) l[n] *= M.fac[n];
          if (i > 0) {
            ok &= wait_all(&M.p_done[(tile - 1) % PB], ((tile - 1) / PB) & 1, abort_f);
            ptx::tc_fence_after();
#pragma unroll
            for (int n = 0; n < 2 * N; n += 16) {
              uint32_t o[16];
              ptx::tmem_ld16(tmem_o + lanes + n, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x)
                o[x] = __float_as_uint(__uint_as_float(o[x]) * M.fac[(n + x) % N]);
              ptx::tmem_st16(tmem_o + lanes + n, o);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
          }
        }
        // P's buffer is free once the product that read it is done
        if (tile >= PB) ok &= wait_all(&M.p_done[tile % PB], ((tile / PB) & 1) ^ 1, abort_f);
        uint8_t* Pb = smem + La::oP + (tile % PB) * La::kP + (j / 64) * (2 * N * 128) + (j % 8) * 2;
        const int ch = (j % 64) / 8;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          if (n < g.t.n_rows) {  // the columns of the other rows are never read
            const float m = M.m[n];
            const float p = exp2_fast(fmaf(s[n], c, m == -INFINITY ? 0.f : -m));
            l[n] += p;
            const bf16 hi = __float2bfloat16_rn(p);
            const bf16 lo = __float2bfloat16_rn(p - __bfloat162float(hi));
            *reinterpret_cast<bf16*>(Pb + n * 128 + ((ch ^ (n & 7)) << 4)) = hi;
            *reinterpret_cast<bf16*>(Pb + (N + n) * 128 + ((ch ^ (n & 7)) << 4)) = lo;
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&M.p_full[tile % PB]);
      }

      // ---- the item, or this CTA's part of it, is done
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (n < g.t.n_rows) {
          const float x = warp_sum(l[n]);
          if (lane == 0) M.red[w][n] = x;
        }
      }
      ok &= wait_all(&M.p_done[(tile - 1) % PB], ((tile - 1) / PB) & 1, abort_f);
      ptx::tc_fence_after();
      named_bar(kBar, 128);
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + g.slot;
      float* part = P.part + slot * N * D;
#pragma unroll
      for (int n0 = 0; n0 < N; n0 += 16) {
        if (n0 >= g.t.n_rows) break;
        uint32_t oh[16], ol[16];
        ptx::tmem_ld16(tmem_o + lanes + n0, oh);
        ptx::tmem_ld16(tmem_o + lanes + N + n0, ol);
        ptx::tmem_ld_wait();
        if (!has_d) continue;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int n = n0 + x;
          if (n >= g.t.n_rows) break;
          const float o = __uint_as_float(oh[x]) + __uint_as_float(ol[x]);
          const float sum = M.red[0][n] + M.red[1][n] + M.red[2][n] + M.red[3][n];
          if (g.parts > 1)
            part[n * D + d] = o;
          else
            write_row<D>(P, g, n, d, o, sum, M.m[n]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&M.o_empty);
        ptx::mbar_arrive(&M.seg_empty[sg % kRing]);
      }
      if (g.parts > 1) {
        for (int n = st_tid; n < g.t.n_rows; n += 128) {
          float* ml = P.part_ml + (slot * N + n) * 2;
          ml[0] = M.m[n];
          ml[1] = M.red[0][n] + M.red[1][n] + M.red[2][n] + M.red[3][n];
        }
        if (last_to_arrive(P, g, g.item, st_tid == 0, &M.last, kBar, 128)) {
          for (int n = st_tid; n < g.t.n_rows; n += 128)
            merged_max<N>(P, g, n, &M.m[n], &M.red[0][n]);
          named_bar(kBar, 128);
          if (has_d) {
            for (int n = 0; n < g.t.n_rows; ++n)
              write_row<D>(P, g, n, d, merged_value<N, D>(P, g, n, d, M.m[n]), M.red[0][n], M.m[n]);
          }
        }
      }
      named_bar(kBar, 128);  // m and red are free
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kCols);
  }
  if (tid == 0 && *abort_f) flag_error(P.err, LORA_DEVERR_TIMEOUT);
}

template <int D, int N>
cudaError_t launch(const CUtensorMap& tm_k, const CUtensorMap& tm_v, AttnParams P, cudaStream_t st,
                   const DeviceInfo& dev) {
  using La = Lay<D, N>;
  constexpr size_t smem = 1024 + La::oMisc + sizeof(Misc<N, La::kStages>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  if (smem > dev.max_smem_optin) return cudaErrorInvalidConfiguration;
  auto kern = attn_decode_kernel<D, N>;
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
  return cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, P);
}

}  // namespace

cudaError_t launch_attn_decode(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                               const AttnParams& P, cudaStream_t st, const DeviceInfo& dev) {
  if (P.kv.head_dim == 64) {
    if (P.rows == 16) return launch<64, 16>(tm_k, tm_v, P, st, dev);
    if (P.rows == 32) return launch<64, 32>(tm_k, tm_v, P, st, dev);
    return launch<64, 64>(tm_k, tm_v, P, st, dev);
  }
  if (P.rows == 16) return launch<128, 16>(tm_k, tm_v, P, st, dev);
  if (P.rows == 32) return launch<128, 32>(tm_k, tm_v, P, st, dev);
  return launch<128, 64>(tm_k, tm_v, P, st, dev);
}

}  // namespace lora
