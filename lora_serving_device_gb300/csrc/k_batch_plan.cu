// A batch's block table, offsets, lengths, slots and positions from the lengths
// of its requests (lora_batch_plan).
//
// Two sums run over the sequences: rows (q_off) and pages (given back, then
// taken); the rest is a lookup a row.  One block makes the sums, kThreads sequences at
// a time, and up to that many leave their ended requests' pages to it too (a warp to a
// request); with more, kernels before and after it count and push them, a warp each over
// the whole GPU (3000 requests, 333 of them ended: 31 us in the one block, 19 us).  Rows are then
// independent: a thread finds its row's sequence in q_off, and its page either in the table or, if
// the page is new, on the stack at the place that the sums give it.  A page's first
// new row writes the page's table entry.
//
// Bound by latency: 20 bytes a sequence and 12 a row (64 single tokens: 4.1 us, of which an
// empty launch takes half).
#include "attn.h"
#include "attn.cuh"

namespace lora {
namespace {

constexpr int kThreads = 1024;
constexpr int kFillThreads = 256;

__device__ __forceinline__ void fill_row(const PlanArgs& a, int t, int n_rows, int top) {
  if (t >= n_rows) {
    if (a.slots != nullptr) a.slots[t] = -1;
    if (a.pos != nullptr) a.pos[t] = -1;
    return;
  }
  int lo = 0, hi = a.n_seqs;  // q_off[lo] <= t < q_off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_off[mid] <= t) lo = mid; else hi = mid;
  }
  const int begin = a.q_off[lo], rows = a.q_off[lo + 1] - begin;
  const int cached = a.kv_len[lo] - rows, p = cached + t - begin;
  const int col = p >> a.lg_page;
  int64_t slot = -1;
  if (col < a.max_pages) {
    int32_t* entry = a.block_table + static_cast<int64_t>(lo) * a.max_pages + col;
    const int have = static_cast<int>((static_cast<int64_t>(cached) + a.page_size - 1) >> a.lg_page);
    int id;
    if (col < have) {
      id = *entry;
    } else {
      const int i = a.take_off[lo] + col - have;
      id = i < top ? a.free_pages[top - 1 - i] : -1;
      // (the page's first position is the first row there: it is past the cached ones)
      if ((p & (a.page_size - 1)) == 0) *entry = id;
    }
    if (id >= 0 && id < a.n_pages)
      slot = static_cast<int64_t>(id) * a.page_size + (p & (a.page_size - 1));
    else
      flag_error(a.err, LORA_DEVERR_BAD_PAGE);
  }
  if (a.slots != nullptr) a.slots[t] = slot;
  if (a.pos != nullptr) a.pos[t] = p;
}

// Inclusive sums over the block of two values; `total` over all threads.
struct Sums {
  int64_t a, b;
};
__device__ __forceinline__ Sums block_scan(Sums x, Sums* warp_sums, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums y = {warp_scan(x.a), warp_scan(x.b)};
  if (lane == 31) warp_sums[warp] = y;
  __syncthreads();
  const Sums w = warp_sums[lane];
  const Sums all = {warp_scan(w.a), warp_scan(w.b)};
  const int before = warp > 0 ? warp - 1 : 0;
  const int64_t ba = __shfl_sync(0xffffffffu, all.a, before), bb = __shfl_sync(0xffffffffu, all.b, before);
  total->a = __shfl_sync(0xffffffffu, all.a, 31);
  total->b = __shfl_sync(0xffffffffu, all.b, 31);
  if (warp > 0) {
    y.a += ba;
    y.b += bb;
  }
  __syncthreads();
  return y;
}

// Pages [from, to) of sequence s's row, by one warp: how many there are (all lanes), and
// onto the stack from place `at` on.
__device__ __forceinline__ int count_pages(const PlanArgs& a, int s, int from, int to) {
  const int32_t* row = a.block_table + static_cast<int64_t>(s) * a.max_pages;
  int n = 0;
#pragma unroll 4
  for (int c = from + (threadIdx.x & 31); c < to; c += 32) n += row[c] >= 0 && row[c] < a.n_pages ? 1 : 0;
  return __reduce_add_sync(0xffffffffu, n);
}
__device__ __forceinline__ void push_pages(const PlanArgs& a, int s, int from, int to, int64_t at) {
  const int lane = threadIdx.x & 31;
  const int32_t* row = a.block_table + static_cast<int64_t>(s) * a.max_pages;
#pragma unroll 4
  for (int c = from; c < to; c += 32) {
    const int id = c + lane < to ? row[c + lane] : -1;
    const bool page = id >= 0 && id < a.n_pages;
    const uint32_t pages = __ballot_sync(0xffffffffu, page);
    const int64_t place = at + __popc(pages & ((1u << lane) - 1u));
    if (page && place < a.free_cap) a.free_pages[place] = id;
    at += __popc(pages);
  }
  if (lane == 0 && at > a.free_cap) flag_error(a.err, LORA_DEVERR_BAD_LEN);
}
// The pages that sequence s holds alone: [from, to) of its row.
__device__ __forceinline__ void own_pages(const PlanArgs& a, int s, int* from, int* to) {
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.lg_page;
  const int64_t cached = min(max(static_cast<int64_t>(a.n_cached[s]), int64_t{0}), cap);
  *from = a.n_shared != nullptr ? max(a.n_shared[s], 0) : 0;
  *to = static_cast<int>((cached + a.page_size - 1) >> a.lg_page);
}

// Of the ended requests, a warp each, before the sums (kPush: after them).
template <bool kPush>
__global__ void __launch_bounds__(kFillThreads) batch_plan_given_kernel(const PlanArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int s = (blockIdx.x * kFillThreads + threadIdx.x) / 32;
  if (s >= a.n_seqs || a.n_new[s] >= 0) return;
  if constexpr (kPush) {
    // (n_cached may have become kv_len: the entries are those that were counted)
    push_pages(a, s, a.span[2 * s], a.span[2 * s + 1], a.give_off[s]);
  } else {
    int from, to;
    own_pages(a, s, &from, &to);
    const int n = count_pages(a, s, from, to);
    if ((threadIdx.x & 31) == 0) {
      a.give[s] = n;
      a.span[2 * s] = from;
      a.span[2 * s + 1] = to;
    }
  }
}

__global__ void __launch_bounds__(kThreads) batch_plan_kernel(const PlanArgs a) {
  __shared__ Sums warp_sums[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  int n_free = *a.n_free;
  if (n_free < 0 || n_free > a.free_cap) {
    if (tid == 0) flag_error(a.err, LORA_DEVERR_BAD_LEN);
    n_free = n_free < 0 ? 0 : a.free_cap;
  }
  int64_t rows_before = 0, taken = 0, given = 0;
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.lg_page;
  for (int s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
    const int s = s0 + tid;
    int64_t cached = 0;
    int fresh = 0, shared = 0;
    if (s < a.n_seqs) {
      cached = a.n_cached[s];
      fresh = a.n_new[s];
      if (a.n_shared != nullptr) shared = max(a.n_shared[s], 0);
    }
    uint32_t bad = 0;
    if (cached < 0 || cached > cap) {
      bad = LORA_DEVERR_BAD_LEN;
      cached = cached < 0 ? 0 : cap;
    }
    const bool ended = fresh < 0;
    Sums total;
    const int64_t rows = ended ? 0 : fresh;
    const Sums r = block_scan({rows, 0}, warp_sums, &total);
    const int64_t T = a.T;
    const int begin = static_cast<int>(min(rows_before + r.a - rows, T));
    const int end = static_cast<int>(min(rows_before + r.a, T));
    rows_before += total.a;
    int64_t len = cached + (end - begin);
    if (end - begin < rows || len > cap) bad = LORA_DEVERR_BAD_LEN;
    const int have = static_cast<int>((cached + a.page_size - 1) >> a.lg_page);
    const int need = static_cast<int>((min(len, cap) + a.page_size - 1) >> a.lg_page);
    const int take = ended ? 0 : need - have;
    int give = 0;
    if (a.apart) {
      if (ended && s < a.n_seqs) give = a.give[s];
    } else {
      // pages of ended requests: a warp counts those of its lanes, one after another
      for (uint32_t left = __ballot_sync(0xffffffffu, ended && have > shared); left != 0;
           left &= left - 1) {
        const int src = __ffs(left) - 1;
        const int from = __shfl_sync(0xffffffffu, shared, src), to = __shfl_sync(0xffffffffu, have, src);
        const int n = count_pages(a, s0 + (tid & ~31) + src, from, to);
        if (lane == src) give = n;
      }
    }
    const Sums p = block_scan({take, give}, warp_sums, &total);
    if (s < a.n_seqs) {
      a.q_off[s] = begin;
      a.kv_len[s] = ended ? 0 : static_cast<int>(min(len, static_cast<int64_t>(INT32_MAX)));
      a.take_off[s] = static_cast<int>(taken + p.a - take);
      if (bad) flag_error(a.err, bad);
    }
    const int64_t first = n_free + given + p.b - give;
    if (a.apart) {
      if (s < a.n_seqs) a.give_off[s] = first;
    } else {
      for (uint32_t left = __ballot_sync(0xffffffffu, give > 0); left != 0; left &= left - 1) {
        const int src = __ffs(left) - 1;
        const int from = __shfl_sync(0xffffffffu, shared, src), to = __shfl_sync(0xffffffffu, have, src);
        push_pages(a, s0 + (tid & ~31) + src, from, to, __shfl_sync(0xffffffffu, first, src));
      }
    }
    taken += total.a;
    given += total.b;
  }
  const int n_rows = static_cast<int>(min(rows_before, static_cast<int64_t>(a.T)));
  const int top = static_cast<int>(min(n_free + given, static_cast<int64_t>(a.free_cap)));
  if (tid == 0) {
    a.q_off[a.n_seqs] = n_rows;
    *a.n_free_out = static_cast<int>(taken < top ? top - taken : 0);
    if (taken > top) flag_error(a.err, LORA_DEVERR_NO_PAGE);
    *a.top = top;
  }
  if (a.fill_here) {
    __syncthreads();
    for (int t = tid; t < a.T; t += kThreads) fill_row(a, t, n_rows, top);
  }
}

__global__ void __launch_bounds__(kFillThreads) batch_plan_fill_kernel(const PlanArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x * kFillThreads + threadIdx.x;
  if (t < a.T) fill_row(a, t, a.q_off[a.n_seqs], *a.top);
}

}  // namespace

cudaError_t launch_batch_plan(const PlanArgs& args, cudaStream_t st) {
  PlanArgs a = args;
  a.fill_here = a.T <= 2 * kThreads;
  a.apart = a.n_seqs > kThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](void (*kernel)(PlanArgs), int blocks, int threads) {
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    return cudaLaunchKernelEx(&cfg, kernel, a);
  };
  const int seq_blocks = (a.n_seqs * 32 + kFillThreads - 1) / kFillThreads;
  cudaError_t e = cudaSuccess;
  if (a.apart) {
    a.fill_here = false;
    e = run(batch_plan_given_kernel<false>, seq_blocks, kFillThreads);
  }
  if (e == cudaSuccess) e = run(batch_plan_kernel, 1, kThreads);
  if (e == cudaSuccess && a.apart) e = run(batch_plan_given_kernel<true>, seq_blocks, kFillThreads);
  if (e == cudaSuccess && !a.fill_here && a.T > 0)
    e = run(batch_plan_fill_kernel, (a.T + kFillThreads - 1) / kFillThreads, kFillThreads);
  return e;
}

}  // namespace lora
