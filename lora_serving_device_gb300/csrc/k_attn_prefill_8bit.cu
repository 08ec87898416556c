// Attention over the 8-bit paged cache for many rows per key head: prompts, chunks
// of prompts and the tokens of a prefix group (lora_attn_paged_8bit and the prefix
// phase of lora_attn_prefix_8bit).
//
// Mathematics, per item (two halves of up to 128 rows of one key head) and key tile of
// 128 keys, for each half:
//   S  = [Q_1 + Q_2] K^T      [128 rows, 128 keys]   e4m3, fp32 in tensor memory
//   s  = c 2^(kb + qb) S      kb, qb the exponents of a key's block and a row
//   P  = 2^(s - m),  l += row sums of P
//   O += P V 2^(vb - R)       [128 rows, D]          f16, P from tensor memory
// K stays as it lies in memory: a row of Q is divided by a power of two and the sum of two
// e4m3 terms, off by at most 2^-17 of its largest value; two products at twice bf16's rate
// take its time.  V would need three terms of P, one and a half times that, so it
// becomes f16 instead: a code is exact there, as is its block's power of two relative to
// the largest so far, R (but for 448 x 2^-25 of that at most), and P keeps 11 bits, where a bf16 has 8.  Four
// warps do it, between the loads and the MMAs; values that no row sees they make zeros on
// the way.  A key block's scale is a factor of its 16 scores beside c.
//
// The bf16 kernel's (k_attn_prefill.cu) schedule of halves, softmax and results, and its floor:
// the tensor cores.  Measured on a warm card: prompt of 8192, 32 / 8 heads of 128: 404 to 413 us (1330 to
// 1360 TFLOP/s, 0.69 to 0.71 of the measured burst rate; 393 in the first moments on a cool one; bf16
// cache 359 to 373); chunks with a window of 1024, 64 / 8 heads of 64: 193 us (117); 8 chunks of 300 behind a
// shared prefix of 8K 333 (306).  The tensor pipe is active for 60% of the cycles, no other pipe for
// more than 35.  A half's chain bounds it, 2400 cycles from scores to weights and 500 back
// through the MMAs, a tile, beside the issuing thread, which is never idle.  The roles
// take more instructions a tile than the bf16 kernel's, so what counted most was to keep them short
// (all 128 scores of a row in registers, one long piece of code: 821 us; loops over 64: 467), the issuing
// thread's commits few (six a tile 467 us, three 433), and Q's split short (429 us, then 419: an
// item's first scores wait for it).
//
// Warps: 0-3 softmax and results of half 0, 4-7 of half 1, 8 schedule and TMA, 9 MMA issue,
// 10 scales, 11 idle, 12-15 Q into its terms and V into f16.  Every wait is bounded; on timeout the kernel
// raises LORA_DEVERR_TIMEOUT.
#include <cudaTypedefs.h>

#include "attn_rows.cuh"

namespace lora {
namespace {

// Four warpgroups, of which two are the softmax's: 160 x 256 + 96 x 256 registers are the
// launch's 128 x 512 (with 128 each, 48 bytes spill: 434 us for 427; so, 24 with blocks of 16 keys).
constexpr int kThreads = 512;
constexpr int kRegsMost = 160, kRegsLeast = 96;
constexpr int kFirstWidener = 12, kWideners = 4;  // warps that widen V
constexpr int kRing = 4;     // segments that the producer may run ahead
// log2 of a row's largest weight when its reference is set, and of the largest that it then lets
// pass: f16 holds 2^15, and what is 2^-30 of the first
constexpr float kTop = 6.f, kMost = 14.f;

template <int D>
struct Lay {
  static constexpr uint32_t kTile = kKeys * D;   // codes of K or V of a tile
  static constexpr uint32_t kWide = 2 * kTile;   // V of a tile in f16; Q's two terms of a half
  static constexpr int kK = D == 128 ? 2 : 4;    // tiles of K in flight
  static constexpr int kV = D == 128 ? 2 : 4;    // of V as codes
  static constexpr int kW = D == 128 ? 3 : 4;    // of V in f16
  static constexpr int kUsed = 4;  // at least kK and kW
  // Buffers of a half's Q: with room for two the next segment's is there before this one's
  // results are written.
  static constexpr int kQ = D == 128 ? 1 : 2;
  // Barriers and scale bytes of a half's Q, a segment each in turn: the softmax warps can come for
  // a segment's when the Qs of kQ later ones are there, and have to find its own.
  static constexpr int kQTurns = 2 * kQ;
  static constexpr uint32_t oV = kK * kTile;
  static constexpr uint32_t oW = oV + kV * kTile;
  static constexpr uint32_t oQ = oW + kW * kWide;
  static constexpr uint32_t oMisc = oQ + 2 * kQ * kWide;  // [half][buffer]
};

template <int D>
struct Misc {
  using La = Lay<D>;
  Segment ring[kRing];
  ScaleRing<2> scales;
  uint64_t k_full[La::kK];
  uint64_t v_full[La::kV], v_empty[La::kV];
  uint64_t w_full[La::kW];
  uint64_t used[La::kUsed];  // Q K^T of a tile and P V of the one before are done
  uint64_t q_in[2][La::kQ], q_empty[2][La::kQ], q_full[2][La::kQTurns];
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2], o_empty[2];
  uint64_t seg_full[kRing], seg_empty[kRing];
  uint8_t q_scale[2][La::kQTurns][kHalf];  // bytes of the rows of Q
  uint32_t tmem;
  int abort;
  int last[2];
};

// V of a tile from codes to f16, the blocks b0, b0 + step, ... by one warp: times 2^(the
// block's exponent - top), in the layout that the MMA reads ([eight keys][64 values][8
// keys][64 values], 128-byte swizzle).  Values that no row sees become zeros.  Eight lanes take
// four 16-code chunks of keys q and q ^ 5: those lie in different halves of the banks
// as codes (by bit 2 or, in rows of 64 bytes, bit 0) and in every other 16 bytes as f16 (by bit 0).
template <int D, int kBlock>
__device__ __forceinline__ void widen_values(const uint8_t* V, uint8_t* W, const uint8_t* bytes,
                                             int top, const RowTile& t, int v0, int b0, int step) {
  constexpr int kHalves = D / 64, kTrips = kBlock / 8 * kHalves;  // eight keys, 64 values a trip
  const int lane = threadIdx.x & 31, c = lane & 3, q = lane >> 3;
  const int r = (lane & 4) != 0 ? q ^ 5 : q;  // key of eight
  const bool edge = tile_has_unseen(t, v0);
  const uint8_t* from = V + r * D + (D == 128 ? c ^ (r & 3) : c ^ (r >> 1)) * 16;
  uint8_t* to = W + r * 128 + ((c * 2 ^ r) << 4);
  uint4 x[kTrips];
  auto read = [&](int b, int k) {
    // the upper four chunks of a row of 128 bytes lie 64 bytes from the lower ones; which come
    // first goes by bit 2 of the key
    const int half = D == 128 ? (((k % kHalves) * 4) ^ (r & 4)) * 16 : 0;
    x[k] = *reinterpret_cast<const uint4*>(from + (b * kBlock + k / kHalves * 8) * D + half);
  };
#pragma unroll
  for (int k = 0; k < kTrips; ++k) read(b0, k);
#pragma unroll 1
  for (int b = b0; b < kKeys / kBlock; b += step) {
    const int e = static_cast<int>(bytes[b]) - top;  // <= 0
    const uint32_t f =
        e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : e >= -24 ? 1u << (24 + e) : 0u;
    const uint32_t f2 = f | f << 16;
#pragma unroll
    for (int k = 0; k < kTrips; ++k) {
      uint4 lo = widen8_e4m3(x[k].x, x[k].y, f2), hi = widen8_e4m3(x[k].z, x[k].w, f2);
      if (b + step < kKeys / kBlock) read(b + step, k);
      if (edge && !place_seen(t, v0 + b * kBlock + k / kHalves * 8 + r)) lo = hi = make_uint4(0, 0, 0, 0);
      uint8_t* at = to + ((b * kBlock / 8 + k / kHalves) * kHalves + k % kHalves) * 1024;
      *reinterpret_cast<uint4*>(at) = lo;
      *reinterpret_cast<uint4*>(W + ((at - W) ^ 16)) = hi;
    }
  }
}

// 32 rows of Q in shared memory, from `row0` on, from bf16 as TMA lays them ([64 values of a
// head][rows][64 values], 128-byte swizzle) to two e4m3 terms in the same place, each 128
// bytes a row (a plane each, or the halves of a row with D = 64), divided by powers of two,
// whose bytes go to `bytes`.  One warp, four lanes to a row: eight rows at once, with a quarter of
// a row's values in a lane, have enough under way that its latencies overlap (16 lanes to a row:
// 5700 cycles, which an item's first scores wait for).
template <int D>
__device__ __forceinline__ void split_queries(uint8_t* Q, int row0, uint8_t* bytes) {
  constexpr int kChunks = D / 32;  // of eight values, of a lane
  constexpr uint32_t kPlane = kHalf * 128;
  const int lane = threadIdx.x & 31, i = lane & 3;
  const uint32_t m = 0x7fff7fffu;
  auto most = [](uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
  };
#pragma unroll 1
  for (int k = 0; k < 32; k += 8) {
    const int row = row0 + k + lane / 4, r = row & 7;
    uint8_t* at = Q + row * 128;
    uint4 x[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int chunk = i * kChunks + c;
      x[c] = *reinterpret_cast<const uint4*>(at + (chunk / 8) * kPlane + (((chunk & 7) ^ r) << 4));
    }
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      top = most(top, most(most(x[c].x & m, x[c].y & m), most(x[c].z & m, x[c].w & m)));
    top = most(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = most(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int byte = min(scale_byte(fmaxf(bf16_lo(top), bf16_hi(top))), 253);
    const float inv = scale_of(254 - byte);
    __syncwarp();  // (the rows have been read)
    const int c0 = i * (kChunks / 2);  // the first 16 codes of a term
#pragma unroll
    for (int c = 0; c < kChunks; c += 2) {
      uint32_t t1[4], t2[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y[8];
        load8(reinterpret_cast<const bf16*>(&x[c + e]), y);
#pragma unroll
        for (int z = 0; z < 2; ++z)
          split4_e4m3(pack_f16x2(y[4 * z] * inv, y[4 * z + 1] * inv),
                      pack_f16x2(y[4 * z + 2] * inv, y[4 * z + 3] * inv), t1[2 * e + z], t2[2 * e + z]);
      }
      const int to = c0 + c / 2;
      *reinterpret_cast<uint4*>(at + ((to ^ r) << 4)) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
      *reinterpret_cast<uint4*>(at + (D == 128 ? kPlane : 0) + (((D == 128 ? to : 4 + to) ^ r) << 4)) =
          make_uint4(t2[0], t2[1], t2[2], t2[3]);
    }
    if (i == 0) bytes[row] = static_cast<uint8_t>(byte);
  }
}

// What a row's scores of a block are multiplied with; never 0, which -infinity would make NaN.
__device__ __forceinline__ float scale_with(float key, float row) {
  return fmaxf(key * row, 1.2e-38f);
}

template <int D, int kBlock>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prefill_8bit_kernel(const __grid_constant__ CUtensorMap tm_q,
                             const __grid_constant__ CUtensorMap tm_k,
                             const __grid_constant__ CUtensorMap tm_v, const AttnParams P) {
  using La = Lay<D>;
  constexpr int kK = La::kK, kV = La::kV, kW = La::kW, kUsed = La::kUsed;
  constexpr int kQ = La::kQ, kQTurns = La::kQTurns;
  using Mi = Misc<D>;
  constexpr uint32_t kIdescQK = ptx::idesc_e4m3_f32(kHalf, kKeys, false, false);
  constexpr uint32_t kIdescPV = ptx::idesc_f16_f32(kHalf, D, false, true);
  constexpr uint32_t kGroupBytes = (D / 64) * 1024;  // eight keys of V in f16

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
    for (int i = 0; i < kK; ++i) {
      ptx::mbar_init(&M.k_full[i], 1);
    }
    for (int i = 0; i < kV; ++i) {
      ptx::mbar_init(&M.v_full[i], 1);
      ptx::mbar_init(&M.v_empty[i], kWideners);
    }
    for (int i = 0; i < kW; ++i) {
      ptx::mbar_init(&M.w_full[i], kWideners);
    }
    for (int i = 0; i < kUsed; ++i) ptx::mbar_init(&M.used[i], 1);
    init_scales(M.scales, 8 + kWideners);
    for (int h = 0; h < 2; ++h) {
      for (int i = 0; i < kQ; ++i) {
        ptx::mbar_init(&M.q_in[h][i], 1);
        ptx::mbar_init(&M.q_empty[h][i], 1);
      }
      for (int i = 0; i < kQTurns; ++i) ptx::mbar_init(&M.q_full[h][i], kWideners);
      ptx::mbar_init(&M.s_full[h], 1);
      ptx::mbar_init(&M.p_half[h], 4);
      ptx::mbar_init(&M.p_full[h], 4);
      ptx::mbar_init(&M.o_done[h], 1);
      ptx::mbar_init(&M.o_empty[h], 4);
    }
    for (int i = 0; i < kRing; ++i) {
      ptx::mbar_init(&M.seg_full[i], 1);
      ptx::mbar_init(&M.seg_empty[i], 10 + kWideners);
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
    TileLoader<D, 1> load(P);
    int nk = 0, nv = 0;     // tiles brought in
    int batches = 0;        // of their scales
    int q_use[2] = {0, 0};  // segments of each half
    bool ok = true;
    SplitItem mine = {};
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
      if (g.n == 0) break;
      bool seen;
      const int id = load.ask(P, g, seen);
      if (P.join_after && g.parts > 1 && g.cta0 == blockIdx.x)
        mine = {g.parts, g.tok0, g.t.row0, g.t.n_rows, g.head, g.shared, {0, 0}};
      for (int h = 0; h < 2 && ok; ++h) {
        if (g.t.n_rows <= h * half_rows) break;
        const int use = q_use[h], buf = use % kQ;
        if (use >= kQ) ok = wait_all(&M.q_empty[h][buf], ((use / kQ) & 1) ^ 1, abort_f);
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&M.q_in[h][buf], half_rows * D * 2);
          for (int x = 0; x < D / 64; ++x)
            tma_load_rows(smem + La::oQ + (h * kQ + buf) * La::kWide + x * (kHalf * 128), &tm_q,
                          &M.q_in[h][buf], g.head * P.group,
                          g.tok0 + P.by_group(g.t.row0 + h * half_rows), x);
        }
        ++q_use[h];
      }
      __syncwarp();
      load.now = load.place(P, g, 0, id, seen);  // (asked for before Q, looked at after)
      for (int i = 0; i < g.n && ok; ++i) {
        const int at = load.at(P, g, i);
        const uint32_t bytes = load.bytes(at);
        if (nk >= kK) ok = wait_all(&M.used[(nk - kK) % kUsed], ((nk - kK) / kUsed) & 1, abort_f);
        if (!ok) break;
        load.load(&tm_k, &M.k_full[nk % kK], smem + nk % kK * La::kTile, at, bytes);
        ++nk;
        if (nv >= kV) ok = wait_all(&M.v_empty[nv % kV], ((nv / kV) & 1) ^ 1, abort_f);
        if (!ok) break;
        load.load(&tm_v, &M.v_full[nv % kV], smem + La::oV + nv % kV * La::kTile, at, bytes);
        ++nv;
      }
    }
    if (P.join_after && lane == 0) P.split[blockIdx.x] = mine;
    if (!ok) {
      // gave up: what is on its way into shared memory has to land first
      int none = 0;
      for (int h = 0; h < 2; ++h)
        for (int k = q_use[h] > kQ ? q_use[h] - kQ : 0; k < q_use[h]; ++k)
          ptx::mbar_wait_bounded(&M.q_in[h][k % kQ], (k / kQ) & 1, &none, kAttnWaitNs / 8);
      for (int k = nk > kK ? nk - kK : 0; k < nk; ++k)
        ptx::mbar_wait_bounded(&M.k_full[k % kK], (k / kK) & 1, &none, kAttnWaitNs / 8);
      for (int k = nv > kV ? nv - kV : 0; k < nv; ++k)
        ptx::mbar_wait_bounded(&M.v_full[k % kV], (k / kV) & 1, &none, kAttnWaitNs / 8);
    }
  } else if (warp == 9) {
    // ---------------- MMA issue ------------------------------------------
    // One thread: P V of a tile, then Q K^T of the next, which takes P's place, half by half,
    // so that the tensor cores have the other half's work while a softmax runs.  A commit
    // takes this thread 150 to 200 cycles, so there are few: scores tell that the product
    // before them is done too, and one a tile frees its K and the V before.
    if (elect_one()) {
      const uint32_t q_tiles = desc_lo(ptx::smem_u32(smem + La::oQ), 16);
      const uint32_t k_tiles = desc_lo(ptx::smem_u32(smem), 16);
      const uint32_t w_tiles = desc_lo(ptx::smem_u32(smem + La::oW), 1024);
      // of each half: the parity of its tiles' P, and its segments so far
      uint32_t p_par = 0;
      int segs0 = 0, segs1 = 0;
      int n = 0;  // tiles
#pragma unroll 1
      for (int sg = 0;; ++sg) {
        wait_quiet(&M.seg_full[sg % kRing], (sg / kRing) & 1, abort_f);
        const int tiles = M.ring[sg % kRing].n, halves = M.ring[sg % kRing].t.n_rows > half_rows ? 2 : 1;
        if (tiles == 0 || *abort_f) break;
#pragma unroll 1
        for (int i = 0; i <= tiles && !*abort_f; ++i, ++n) {
          const int w_at = (n - 1) % kW, k_at = n % kK;
#pragma unroll 1
          for (int h = 0; h < halves; ++h) {
            const uint32_t tm_s = tmem + h * 128, tm_o = tmem + 256 + h * 128;
            const int use = h == 0 ? segs0 : segs1;
            if (i > 0) {
              const uint32_t va = w_tiles + w_at * (La::kWide / 16);
              if (h == 0) wait_quiet(&M.w_full[w_at], ((n - 1) / kW) & 1, abort_f);
              // the half's previous segment has been read out of O
              if (i == 1 && use > 0) wait_quiet(&M.o_empty[h], (use & 1) ^ 1, abort_f);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                wait_quiet(x ? &M.p_full[h] : &M.p_half[h], (p_par >> h) & 1, abort_f);
                ptx::tc_fence_after();
#pragma unroll
                for (int ks = 4 * x; ks < 4 * x + 4; ++ks)
                  mma_ts(tm_o, tm_s + ks * 8, va + ks * 2 * kGroupBytes / 16,
                         desc_hi(kGroupBytes), kIdescPV, ks > 0 || i > 1 ? 1u : 0u);
              }
              p_par ^= 1u << h;
            }
            if (i < tiles) {
              const uint32_t qa = q_tiles + (h * kQ + use % kQ) * (La::kWide / 16), ka = k_tiles + k_at * (La::kTile / 16);
              if (i == 0) wait_quiet(&M.q_full[h][use % kQTurns], (use / kQTurns) & 1, abort_f);
              if (h == 0) wait_quiet(&M.k_full[k_at], (n / kK) & 1, abort_f);
              ptx::tc_fence_after();
#pragma unroll
              for (int ks = 0; ks < 2 * D / 32; ++ks)  // both terms of Q against the same keys
                mma_ss_8bit(tm_s, qa + ((ks / 4) * (kHalf * 128) + (ks % 4) * 32) / 16,
                            desc_hi(1024), ka + ks % (D / 32) * 2, desc_hi_span(8 * D, D),
                            kIdescQK, ks > 0 ? 1u : 0u);
              ptx::mma_commit(&M.s_full[h]);
              if (i == tiles - 1) ptx::mma_commit(&M.q_empty[h][use % kQ]);
            } else {
              ptx::mma_commit(&M.o_done[h]);
              if (h == 0) ++segs0; else ++segs1;
            }
          }
          if (i < tiles) ptx::mma_commit(&M.used[n % kUsed]);
        }
        --n;
        ptx::mbar_arrive(&M.seg_empty[sg % kRing]);
      }
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---------------- scales ----------------------------------------------
    run_scales(P, M.scales, M.ring, kRing, M.seg_full, M.seg_empty, abort_f);
  } else if (warp >= kFirstWidener) {
    // ---------------- Q into terms, V from codes to f16 --------------------
    const ScaleReader scales(P);
    bool ok = true;
    int n = 0, q_use[2] = {0, 0};
    for (int sg = 0; ok; ++sg) {
      ok = wait_all(&M.seg_full[sg % kRing], (sg / kRing) & 1, abort_f);
      if (!ok) break;
      const Segment& g = M.ring[sg % kRing];
      if (g.n == 0) break;
      // Q first, beside the softmax warps' results of the segment before
#pragma unroll 1
      for (int h = 0; h < 2 && ok && g.t.n_rows > h * half_rows; ++h) {
        const int use = q_use[h], buf = use % kQ;
        ok = wait_all(&M.q_in[h][buf], (use / kQ) & 1, abort_f);
        split_queries<D>(smem + La::oQ + (h * kQ + buf) * La::kWide, (warp - kFirstWidener) * 32,
                         M.q_scale[h][use % kQTurns]);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&M.q_full[h][use % kQTurns]);
        ++q_use[h];
      }
      for (int i = 0; i < g.n && ok; ++i, ++n) {
        const int sc = scales.of(M.scales, g, i, abort_f);
        ok = wait_all(&M.v_full[n % kV], (n / kV) & 1, abort_f) &&
             (n < kW || wait_all(&M.used[(n - kW + 1) % kUsed], ((n - kW + 1) / kUsed) & 1, abort_f));
        if (!ok) break;
        widen_values<D, kBlock>(smem + La::oV + n % kV * La::kTile, smem + La::oW + n % kW * La::kWide,
                                M.scales.v[sc], M.scales.top[sc], g.t, (g.first + i) * kKeys,
                                warp - kFirstWidener, kWideners);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&M.w_full[n % kW]);
          ptx::mbar_arrive(&M.v_empty[n % kV]);
        }
        scales.done(M.scales, g, i);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&M.seg_empty[sg % kRing]);
    }
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
    const ScaleReader scales(P);
    int tile = 0, segs = 0;  // tiles and segments of this half so far
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
      const int min_hi = __reduce_min_sync(0xffffffffu, hi), max_lo = __reduce_max_sync(0xffffffffu, lo);
      // (this half may have left out segments, and with them batches of scales: the warps that split Q
      // have used them all before)
      wait_quiet(&M.q_full[h][segs % kQTurns], (segs / kQTurns) & 1, abort_f);
      const float q_scale = c * scale_of(M.q_scale[h][segs % kQTurns][row]);
      ++segs;
      const int readers = g.t.n_rows <= half_rows ? 2 : 1;  // the other half's warp too, if it has no rows
      float m = -INFINITY, l = 0.f;  // m: what weights are relative to
      int R = 0;                     // the largest exponent of a value block so far
#pragma unroll 1
      for (int i = 0; i < g.n; ++i, ++tile) {
        const int v0 = (g.first + i) * kKeys, key0 = window_key(g.t, v0);  // place, key
        const int sc = scales.of(M.scales, g, i, abort_f);
        const float* key_scale = M.scales.k[sc];
        const int top = M.scales.top[sc];
        wait_quiet(&M.s_full[h], tile & 1, abort_f);
        __syncwarp();
        ptx::tc_fence_after();
        if (key0 + kKeys - 1 > min_hi || key0 < max_lo)
          mask_in_place(tm_s, key0, hi, lo, min(g.t.n_sink, hi + 1) - v0);
        // (the scores are read twice: here for the largest of each block, all at once: prompt of
        // 8192 400 us, 64 keys at a time 405; with a window 193 and 196; blocks of 8 keys
        // have twice the maxima, more than the registers hold, and keep to 64 keys)
        constexpr int kTops = kBlock == 16 ? kKeys : 64;
        float mx = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < kKeys; k += kTops) {
          float s[kTops / kBlock][kBlock], top_s[kTops / kBlock];
#pragma unroll
          for (int b = 0; b < kTops / kBlock; ++b) ptx::tmem_ld_top(tm_s + k + b * kBlock, s[b], top_s[b]);
          float kc[kTops / kBlock];  // (read beside the scores)
#pragma unroll
          for (int b = 0; b < kTops / kBlock; ++b) kc[b] = scale_with(key_scale[k / kBlock + b], q_scale);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int b = 0; b < kTops / kBlock; ++b) mx = fmaxf(mx, top_s[b] * kc[b]);
        }
        // (rows that are not in use hold anything: they have no say)
        if (top > R || __any_sync(0xffffffffu, mine && mx > m + kMost)) {
          const float now = fmaxf(m, mx - kTop);
          const float f = m == -INFINITY ? 0.f : exp2_fast(m - now);
          m = now;
          l *= f;
          const float f_all = top - R < 127 ? f * scale_of(127 - (top - R)) : 0.f;
          R = top;
          if (i > 0) {
            // (the product before these scores is done)
            scale_result<D>(tm_o, f_all);
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        const uint64_t neg2 = pack2(neg, neg);
        uint64_t sum0 = 0, sum1 = 0;
#pragma unroll 1
        for (int k = 0; k < kKeys; k += 64) {
          float s[64];
          ptx::tmem_ld32(tm_s + k, *reinterpret_cast<uint32_t(*)[32]>(s));
          ptx::tmem_ld32(tm_s + k + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
          float key_c[64 / kBlock];
#pragma unroll
          for (int b = 0; b < 64 / kBlock; ++b) key_c[b] = scale_with(key_scale[k / kBlock + b], q_scale);
          ptx::tmem_ld_wait();
          uint32_t p[32];
#pragma unroll
          for (int b = 0; b < 64 / kBlock; ++b) {
            const uint64_t kc2 = pack2(key_c[b], key_c[b]);
#pragma unroll
            for (int x = b * kBlock; x < (b + 1) * kBlock; x += 2) {
              float e0, e1;
              unpack2(fma2(pack2(s[x], s[x + 1]), kc2, neg2), &e0, &e1);
              e0 = exp2_fast(e0);
              e1 = exp2_fast(e1);
              if (x & 2)
                sum1 = add2(sum1, pack2(e0, e1));
              else
                sum0 = add2(sum0, pack2(e0, e1));
              p[x / 2] = pack_f16x2(e0, e1);
            }
          }
          ptx::tmem_st32(tm_s + k / 2, p);
          // each half of the keys goes to the MMA as soon as it is there
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(k == 0 ? &M.p_half[h] : &M.p_full[h]);
        }
        scales.done(M.scales, g, i, readers);
        float a, b;
        unpack2(add2(sum0, sum1), &a, &b);
        l += a + b;
      }

      // ---- the item, or this CTA's part of it, is done
      finish_half<D, true>(P, g, h, row, mine, g.tok0 + tok, head, m, l, scale_of(max(R, 1)), tm_o, &M.o_done[h],
                     (segs - 1) & 1, abort_f, &M.o_empty[h], &M.seg_empty[sg % kRing], &M.last[h], bar);
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

template <int D, int kBlock>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnParams& P,
                   cudaStream_t st, const DeviceInfo& dev) {
  using La = Lay<D>;
  constexpr size_t smem = 1024 + La::oMisc + sizeof(Misc<D>);
  static_assert(smem <= 232448, "shared memory of a CTA");
  if (smem > dev.max_smem_optin) return cudaErrorInvalidConfiguration;
  auto kern = attn_prefill_8bit_kernel<D, kBlock>;
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

cudaError_t launch_attn_prefill_8bit(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                     const CUtensorMap& tm_v, const AttnParams& P,
                                     cudaStream_t st, const DeviceInfo& dev) {
  if (P.kv.page_size == 8)
    return P.kv.head_dim == 64 ? launch<64, 8>(tm_q, tm_k, tm_v, P, st, dev)
                               : launch<128, 8>(tm_q, tm_k, tm_v, P, st, dev);
  return P.kv.head_dim == 64 ? launch<64, 16>(tm_q, tm_k, tm_v, P, st, dev)
                             : launch<128, 16>(tm_q, tm_k, tm_v, P, st, dev);
}

}  // namespace lora
