// Device helpers shared by the paged-cache kernels: finding a row's sequence,
// and the schedule of the attention kernels.
//
// The schedule.  A problem is a run of consecutive tokens that attend to one
// block-table row over the keys [k_lo, k_hi): a sequence, or a prefix group
// (all its sequences' tokens against the shared prefix).  Its rows, (token,
// query head of one key head), are packed token-major and cut into row tiles
// of P.rows; a row tile sees some 128-key tiles.  An item is (row tile, key
// head); its units are its key tiles, after P.over units that stand for the
// cost of taking it up and finishing it.  All units, numbered row tile by row
// tile, key head by key head, are cut into equal contiguous shares, one per
// CTA, whatever the lengths are (they live on the device).  An item that
// several CTAs share (short ones are not shared) is finished by the last of
// them to arrive, or by a kernel after them; either adds the parts in CTA
// order, so the result is a function of the lengths alone.
// Each CTA finds its share itself: its threads size a problem each, and one
// warp adds the sizes up and looks for its place.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace lora {

// The sequence that row t of the batch belongs to: the largest s with
// q_off[s] <= t, found by the whole warp in log32(n_seqs) loads; -1 for rows
// of no sequence.  Sequences without new tokens are skipped by taking the
// largest.
__device__ __forceinline__ int seq_of_row(const int32_t* q_off, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n_seqs;  // q_off[lo] <= t assumed; the answer is in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;
    const bool le = i <= hi && q_off[i] <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    const int new_lo = lo + n * step;
    const int new_hi = new_lo + step - 1;
    lo = new_lo;
    hi = new_hi < hi ? new_hi : hi;
  }
  return lo < n_seqs && q_off[0] <= t ? lo : -1;
}

constexpr int kKeys = 128;     // keys of a tile

// n / d for 0 <= n < 2^31 by a multiplication: with s = ceil(log2 d) and mul =
// floor(2^(31+s) / d) + 1 the product exceeds n 2^(31+s) / d by less than
// 2^(31+s) / d.
struct FastDiv {
  uint32_t mul;
  int shift;
  static FastDiv of(int d) {
    int s = 0;
    while ((int64_t{1} << s) < d) ++s;
    return {static_cast<uint32_t>((uint64_t{1} << (31 + s)) / d + 1), 31 + s};
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul >> shift);
  }
};

// An item that several CTAs share, from the one it begins in.
struct SplitItem {
  int parts;          // 0: there is none
  int tok0, row0, n_rows;
  int head, shared;
  int pad[2];
};

struct AttnParams {
  lora_paged_kv_t kv;
  const bf16* q;
  int64_t q_stride, out_stride;
  bf16* out;
  const int32_t *group_off, *prefix_len;
  int n_groups;
  bool groups_phase;   // problems are the prefix groups (else the sequences)
  int group;           // query heads of a key head
  int rows;            // rows of a row tile
  FastDiv by_group, by_rows;
  int lg_page;         // log2 of the page size
  int box;             // rows of a page that are loaded at once
  int over;            // units that an item costs beside its key tiles
  int whole;           // items of up to that many key tiles are not split
  bool join_after;     // parts are joined by a kernel of their own (prefill)
  int n_q_heads;
  float scale_log2;    // scale * log2(e)
  int window, n_sink;
  uint32_t* err;
  uint32_t* count;     // [CTA][2] arrivals of the (halves of the) item that begins there
                       // and ends in another; zero between calls
  float* part;         // [CTA][2][row tile] partial sums
  float* part_ml;      // [CTA][2][rows][2] their maxima (log2 units) and sums
  SplitItem* split;    // [CTA] the item that begins there and ends in another (prefill)
  float* prior;        // [T][n_q_heads][D] the prefix phase's result, fp32
  float* prior_lse;    // [T][n_q_heads] its log2-sum-exp
  const uint8_t *k_scale, *v_scale;  // of a cache in 8 bits, or null
  int scale_tiles;     // key tiles whose scales are looked up at once
};

// One problem.
struct Problem {
  int tok0, n_rows;    // first token, rows over all row tiles
  int base;            // position of the first token (sequences)
  int k_lo, k_hi;
  int table_row;
};

// One row tile's view.  Keys [vis_lo, vis_hi] and the first n_sink are those
// that some row sees.  Its key tiles run over them closed up, in whole boxes:
// place v is key v below sink_places and key origin + v - sink_places from there
// on, tile i is places [128 i, 128 i + 128).  n_tiles >= 1 unless the row tile
// has nothing to write.
struct RowTile {
  int row0, n_rows;
  int vis_lo, vis_hi, n_sink;
  int sink_places, origin, n_tiles;
};

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) {
  return x < lo ? lo : x > hi ? hi : x;
}

// The first position in the window of a row at `pos`.  (Compared before the
// subtraction, which overflows for a row before position 0 and the widest
// windows.)
__device__ __forceinline__ int window_first(const AttnParams& P, int pos) {
  return P.window > 0 && pos >= P.window ? pos - P.window + 1 : 0;
}

// The group of sequence s (0 .. n_groups - 1), or -1.
__device__ __forceinline__ int group_of_seq(const AttnParams& P, int s) {
  const int n = P.n_groups;
  if (n <= 16) {  // loads that do not wait for one another
    int g = -1;
#pragma unroll 4
    for (int i = 0; i <= n; ++i) g += P.group_off[i] <= s ? 1 : 0;
    return g < n ? g : -1;
  }
  int lo = 0, hi = n;  // group_off[lo] <= s < group_off[hi], if in any
  if (s < P.group_off[lo] || s >= P.group_off[hi]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (P.group_off[mid] <= s) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int key_cap(const AttnParams& P) { return P.kv.max_pages * P.kv.page_size; }

// Positions [0, shared_keys) of sequence s are attended in the prefix phase.
__device__ __forceinline__ int shared_keys(const AttnParams& P, int s) {
  if (P.n_groups == 0) return 0;
  const int g = group_of_seq(P, s);
  return g < 0 ? 0 : clamp_int(P.prefix_len[g], 0, key_cap(P));
}

// Tokens [*t0, *t1) of problem p.
__device__ __forceinline__ void problem_tokens(const AttnParams& P, int p, int* t0, int* t1) {
  int s0 = p, s1 = p + 1;
  if (P.groups_phase) {
    s0 = P.group_off[p], s1 = P.group_off[p + 1];
    if (s0 < 0 || s1 < s0 || s1 > P.kv.n_seqs) {
      flag_error(P.err, LORA_DEVERR_BAD_LEN);
      *t0 = *t1 = 0;
      return;
    }
    if (P.prefix_len[p] <= 0) s1 = s0;
  }
  int a = P.kv.q_off[s0], b = P.kv.q_off[s1];
  if (a < 0 || b < a || b > P.kv.T) {
    flag_error(P.err, LORA_DEVERR_BAD_LEN);
    a = b = 0;
  }
  *t0 = a;
  *t1 = b;
}

__device__ __forceinline__ Problem load_problem(const AttnParams& P, int p) {
  Problem r;
  int b;
  problem_tokens(P, p, &r.tok0, &b);
  r.n_rows = (b - r.tok0) * P.group;
  const int cap = key_cap(P);
  if (P.groups_phase) {
    r.table_row = P.group_off[p];
    r.base = 0;
    r.k_lo = 0;
    r.k_hi = P.prefix_len[p];
    if (r.k_hi > cap) {
      flag_error(P.err, LORA_DEVERR_BAD_LEN);
      r.k_hi = cap;
    }
    return r;
  }
  r.table_row = p;
  int len = P.kv.kv_len[p];
  if (len > cap) {
    flag_error(P.err, LORA_DEVERR_BAD_LEN);
    len = cap;
  }
  len = len < -(1 << 24) ? -(1 << 24) : len;
  r.base = len - (b - r.tok0);
  r.k_lo = shared_keys(P, p);
  if (r.k_lo > 0 && b > r.tok0 && r.k_lo > r.base) flag_error(P.err, LORA_DEVERR_BAD_LEN);
  r.k_hi = len;
  return r;
}

__device__ __forceinline__ RowTile row_tile(const AttnParams& P, const Problem& pr, int rt) {
  RowTile t;
  t.row0 = rt * P.rows;
  t.n_rows = min(P.rows, pr.n_rows - t.row0);
  if (P.groups_phase) {
    t.vis_lo = 0;
    t.vis_hi = pr.k_hi - 1;
    t.n_sink = t.sink_places = t.origin = 0;
    t.n_tiles = (pr.k_hi + kKeys - 1) / kKeys;
    return t;
  }
  const int first = pr.base + P.by_group(t.row0);
  t.vis_hi = min(pr.base + P.by_group(t.row0 + t.n_rows - 1), pr.k_hi - 1);
  t.vis_lo = max(window_first(P, first), pr.k_lo);
  t.n_sink = P.window > 0 ? max(min(P.n_sink, t.vis_hi + 1), 0) : 0;
  t.sink_places = (t.n_sink + P.box - 1) & -P.box;
  t.origin = t.vis_lo & -P.box;
  if (t.sink_places > t.origin) t.sink_places = t.origin = 0;  // they meet: one run from key 0
  t.n_tiles = (t.sink_places + max(t.vis_hi - t.origin + 1, 0) + kKeys - 1) / kKeys;
  if (t.n_tiles < 1) t.n_tiles = 1;
  return t;
}

// The key at place v, if v is not one of the first tokens' places (there it is
// below origin, and so below what any row's window begins with).
__device__ __forceinline__ int window_key(const RowTile& t, int v) {
  return t.origin + v - t.sink_places;
}

// What a CTA does next: key tiles [tile0, tile0 + n) of an item.
struct Segment {
  int n;             // key tiles; 0: the CTA is done
  int first;         // the item's number of the first of them
  int head;          // key head
  int table_row, tok0, base, k_lo;
  int shared;        // the rows have a prior part from the prefix phase
  RowTile t;
  int cta0, parts;   // the CTAs that share the item: cta0 .. cta0 + parts - 1
  int tile0;         // key tiles of this CTA before the segment
  int batch0;        // batches of P.scale_tiles key tiles before it (a cache in 8 bits)
  int once;          // no other CTA reads these key tiles
  int slot;          // where this CTA's part goes, if parts > 1
};

// Units of one key head over all row tiles of a problem: a warp's lanes take a
// row tile each.
__device__ __forceinline__ int64_t problem_units(const AttnParams& P, const Problem& pr) {
  const int n = P.by_rows(pr.n_rows + P.rows - 1);
  int64_t sum = 0;
  for (int rt = threadIdx.x & 31; rt < n; rt += 32) sum += row_tile(P, pr, rt).n_tiles + P.over;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Sizes of the first kSized problems: row tiles and units of one key head (-1
// units: not added up yet, many row tiles).  All threads of the CTA compute
// them, into shared memory that the first tiles will overwrite.
constexpr int kSized = 2048;
struct ProblemSize {
  int tiles, units;
};
__device__ __forceinline__ ProblemSize problem_size(const AttnParams& P, const Problem& pr) {
  ProblemSize z;
  z.tiles = P.by_rows(pr.n_rows + P.rows - 1);
  z.units = z.tiles > 4 ? -1 : 0;
  if (z.tiles <= 4)
    for (int rt = 0; rt < z.tiles; ++rt) z.units += row_tile(P, pr, rt).n_tiles + P.over;
  return z;
}
// All threads; the caller follows it with a barrier.
__device__ __forceinline__ void size_problems(const AttnParams& P, ProblemSize* sizes) {
  const int n = min(P.groups_phase ? P.n_groups : P.kv.n_seqs, kSized);
  for (int p = threadIdx.x; p < n; p += blockDim.x) sizes[p] = problem_size(P, load_problem(P, p));
}

// After it and a barrier, the long ones: a warp to a problem.
__device__ __forceinline__ void size_long_problems(const AttnParams& P, ProblemSize* sizes) {
  const int n = min(P.groups_phase ? P.n_groups : P.kv.n_seqs, kSized);
  for (int p = threadIdx.x / 32; p < n; p += blockDim.x / 32) {
    if (sizes[p].units >= 0) continue;
    const int64_t units = problem_units(P, load_problem(P, p));
    __syncwarp();
    if ((threadIdx.x & 31) == 0 && units <= INT32_MAX) sizes[p].units = static_cast<int>(units);
  }
}

// 32 consecutive problems, one to a lane.  Those of many row tiles (prompts)
// are added up by the whole warp.
struct LaneSize {
  int tiles;
  int64_t units;
};
__device__ __forceinline__ LaneSize lane_sizes(const AttnParams& P, ProblemSize* sizes, int p0,
                                               int n_prob) {
  const int lane = threadIdx.x & 31, p = p0 + lane;
  ProblemSize z = {0, 0};
  if (p < n_prob) z = p0 < kSized ? sizes[p] : problem_size(P, load_problem(P, p));
  LaneSize r = {z.tiles, z.units};
  for (uint32_t many = __ballot_sync(0xffffffffu, z.units < 0); many != 0; many &= many - 1) {
    const int src = __ffs(many) - 1;
    const int64_t all = problem_units(P, load_problem(P, p0 + src));
    if (lane == src) {
      r.units = all;
      if (p0 < kSized && all <= INT32_MAX) sizes[p].units = static_cast<int>(all);
    }
  }
  return r;
}
template <typename T>
__device__ __forceinline__ T warp_total(T x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <typename T>
__device__ __forceinline__ T warp_scan(T x) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  return x;
}

// Walks a CTA's share (one warp, all lanes alike).
struct Walker {
  Problem pr;
  RowTile t;
  int prob, rt;      // the problem, and the row tile's number in it
  int u, begin, end; // next unit, the share's
  int total, share;  // units of the call, units of a CTA
  int tile_unit;     // first unit of the row tile
  int done;          // key tiles of the segments so far
  int n_prob;

  __device__ __forceinline__ int units(const AttnParams& P) const {  // of the row tile
    return (t.n_tiles + P.over) * P.kv.n_kv_heads;
  }
  // `sizes`: see size_problems; not used after this.
  __device__ __forceinline__ void start(const AttnParams& P, ProblemSize* sizes) {
    const int hk = P.kv.n_kv_heads, lane = threadIdx.x & 31;
    n_prob = P.groups_phase ? P.n_groups : P.kv.n_seqs;
    done = 0;
    // the sizes of all problems, then the equal share of a CTA
    int64_t units = 0, items = 0;
    for (int p0 = 0; p0 < n_prob; p0 += 32) {
      const LaneSize x = lane_sizes(P, sizes, p0, n_prob);
      units += x.units;
      items += x.tiles;
    }
    __syncwarp();
    units = warp_total(units) * hk;
    items = warp_total(items) * hk;
    // more units than a call could ever work off (2^31 of them read 10^14
    // bytes): refused
    const bool ok = units <= INT32_MAX;
    if (!ok) flag_error(P.err, LORA_DEVERR_BAD_LEN);
    total = ok ? static_cast<int>(units) : 0;
    // Equal shares, but an item of a few key tiles is not worth splitting, nor
    // is less than four tiles worth a CTA.
    const int even = static_cast<int>((static_cast<uint32_t>(total) + gridDim.x - 1) / gridDim.x);
    const int span = ok && items > 0 ? static_cast<int>((units + items - 1) / items) : 1;
    const int least = span <= 8 ? span : 4;
    share = even > least ? even : least;
    const int64_t first = static_cast<int64_t>(share) * blockIdx.x;
    u = first < total ? static_cast<int>(first) : total;
    begin = u;
    end = total - u < share ? total : u + share;
    if (u >= end) return;
    // the problem that unit u belongs to
    tile_unit = 0;
    for (int p0 = 0;; p0 += 32) {
      const LaneSize x = lane_sizes(P, sizes, p0, n_prob);
      const int own = static_cast<int>(x.units) * hk, incl = warp_scan(own);
      const uint32_t past = __ballot_sync(0xffffffffu, tile_unit + incl > u);
      if (past != 0) {
        const int k = __ffs(past) - 1;
        prob = p0 + k;
        tile_unit += __shfl_sync(0xffffffffu, incl - own, k);
        break;
      }
      tile_unit += __shfl_sync(0xffffffffu, incl, 31);
    }
    pr = load_problem(P, prob);
    // the row tile in it, 32 at a time
    const int n = P.by_rows(pr.n_rows + P.rows - 1);
    rt = 0;
    if (n > 1) {
      for (;; rt += 32) {
        const int own = rt + lane < n ? (row_tile(P, pr, rt + lane).n_tiles + P.over) * hk : 0;
        const int incl = warp_scan(own);
        const uint32_t past = __ballot_sync(0xffffffffu, tile_unit + incl > u);
        if (past != 0) {
          const int k = __ffs(past) - 1;
          tile_unit += __shfl_sync(0xffffffffu, incl - own, k);
          rt += k;
          break;
        }
        tile_unit += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    t = row_tile(P, pr, rt);
  }
  // The next row tile; there is one while u is below the total.
  __device__ __forceinline__ void advance(const AttnParams& P) {
    tile_unit += units(P);
    ++rt;
    if (rt * P.rows >= pr.n_rows) {
      rt = 0;
      do {
        ++prob;
        pr = load_problem(P, prob);
      } while (pr.n_rows == 0 && prob + 1 < n_prob);
    }
    t = row_tile(P, pr, rt);
  }
  __device__ __forceinline__ Segment next(const AttnParams& P) {
    Segment g;
    g.n = 0;
    int a, b;
    for (;;) {
      if (u >= end) return g;
      while (tile_unit + units(P) <= u) advance(P);
      const int span = t.n_tiles + P.over;
      g.head = (u - tile_unit) / span;
      a = tile_unit + g.head * span + P.over;
      b = a + t.n_tiles;
      if (t.n_tiles <= P.whole) {
        // a short item goes whole to the CTA that its first unit falls to
        u = b;
        if (a - P.over < begin) continue;
        g.first = 0;
        g.n = t.n_tiles;
        break;
      }
      if (u < a) u = a;
      if (u >= end) return g;  // the share ends in front of the item's key tiles
      g.first = u - a;
      g.n = (end < b ? end : b) - u;
      u += g.n;
      break;
    }
    g.table_row = pr.table_row;
    g.tok0 = pr.tok0;
    g.base = pr.base;
    g.k_lo = pr.k_lo;
    g.shared = pr.k_lo > 0 ? 1 : 0;
    g.t = t;
    // (only key tiles make a CTA one of the item's)
    g.cta0 = blockIdx.x;
    g.parts = 1;
    if (g.n < t.n_tiles) {
      g.cta0 = a / share;
      g.parts = (b - 1) / share - g.cta0 + 1;
    }
    g.slot = blockIdx.x == g.cta0 ? 1 : 0;
    g.tile0 = done;
    g.once = pr.n_rows <= P.rows ? 1 : 0;
    done += g.n;
    return g;
  }
};

}  // namespace lora
