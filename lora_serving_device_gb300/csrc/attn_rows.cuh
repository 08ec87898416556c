// Parts that the attention kernels with rows in the MMA's M share (a thread owns a row):
// masks, rescaling, and the ends of items.
#pragma once

#include "attn.cuh"
#include "attn_tile.cuh"
#include "ptx.cuh"

namespace lora {

constexpr int kHalf = 128;   // rows of a half in the MMA

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t x, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The lowest n bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Part of a row tile, [slot][half][D / 4][128 rows][4]: neighbouring threads
// (rows) write neighbouring vectors.
template <int D>
__device__ __forceinline__ float4* part_row(const AttnParams& P, int64_t slot, int half, int row) {
  return reinterpret_cast<float4*>(P.part) + (slot * 2 + half) * (D / 4) * kHalf + row;
}

// The scores of a tile's keys that a row does not see become -infinity: it sees those from lo
// to hi, key0 being the tile's first, and the tile's first `first`.  A warp's rows, a
// lane each, in tensor memory, by a loop; whether there were any.
__device__ __forceinline__ bool mask_in_place(uint32_t tm_s, int key0, int hi, int lo, int first) {
  if (!__any_sync(0xffffffffu, key0 + kKeys - 1 > hi || key0 < lo)) return false;
#pragma unroll 1
  for (int k = 0; k < kKeys; k += 32) {
    const uint32_t seen = (low_bits(hi + 1 - key0 - k) & ~low_bits(lo - key0 - k)) |
                          low_bits(first - k);
    if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
    uint32_t x[32];
    ptx::tmem_ld32(tm_s + k, x);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int y = 0; y < 32; ++y)
      if (!(seen & (1u << y))) x[y] = 0xff800000u;  // -infinity
    ptx::tmem_st32(tm_s + k, x);
  }
  ptx::tmem_st_wait();
  return true;
}
// The same for scores that have been read already: read again, since changing them in
// registers takes 5 KB of instructions (prompt of 4000, 64 values a head: 182 : 167 us).
__device__ __forceinline__ void mask_scores(uint32_t tm_s, int key0, int hi, int lo, int first,
                                            float (&s)[kKeys]) {
  if (!mask_in_place(tm_s, key0, hi, lo, first)) return;
#pragma unroll
  for (int k = 0; k < kKeys; k += 32)
    ptx::tmem_ld32(tm_s + k, *reinterpret_cast<uint32_t(*)[32]>(s + k));
  ptx::tmem_ld_wait();
}

// A row's result in tensor memory times f.
template <int D>
__device__ __forceinline__ void scale_result(uint32_t tm_o, float f) {
#pragma unroll 1
  for (int k = 0; k < D; k += 32) {
    uint32_t o[32];
    ptx::tmem_ld32(tm_o + k, o);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
    ptx::tmem_st32(tm_o + k, o);
  }
}

// The end of an item, or of this CTA's part of it, for half h: a thread's row (token t, query
// head `head`; `mine`: it is in use) leaves tensor memory, `unit` times what is there, at
// maximum m (log2 units) and sum l.  Rows that several CTAs share are written as
// parts and joined by the last CTA to arrive, or by a kernel after this one.  The last product
// is waited for here (o_done).  kRolled: by short loops, in few registers.
template <int D, bool kRolled = false>
__device__ __forceinline__ void finish_half(const AttnParams& P, const Segment& g, int h, int row,
                                            bool mine, int64_t t, int head, float m, float l,
                                            float unit, uint32_t tm_o, uint64_t* o_done,
                                            uint32_t parity, volatile int* abort,
                                            uint64_t* o_empty, uint64_t* seg_empty, int* last,
                                            int bar) {
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + g.slot;
  RowWriter<D> out(P, g.shared, t, head, mine && g.parts == 1, m, l);
  const RowUnit by(unit);
  out.own *= by.factor;
  wait_quiet(o_done, parity, abort);
  __syncwarp();
  ptx::tc_fence_after();
  auto read = [&] {  // O has been read
    ptx::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      ptx::mbar_arrive(o_empty);
      ptx::mbar_arrive(seg_empty);
    }
  };
  if (g.parts == 1) {
    // (rolled, for the instructions' sake: chunks with a window of 1024 117 us,
    // unrolled 121)
#pragma unroll 1
    for (int k = 0; k < D; k += 16) {
      float o[16];
      ptx::tmem_ld16(tm_o + k, *reinterpret_cast<uint32_t(*)[16]>(o));
      ptx::tmem_ld_wait();
#pragma unroll
      for (int x = 0; x < 16; ++x) o[x] *= by.first;
      if (mine) out.write16(k, o);
    }
    read();
    return;
  }
  if constexpr (kRolled) {
    float2* ml = reinterpret_cast<float2*>(P.part_ml) + h * kHalf + row;
    const PartScale part(l);
#pragma unroll 1
    for (int k = 0; k < D; k += 16) {
      float o[16];
      ptx::tmem_ld16(tm_o + k, *reinterpret_cast<uint32_t(*)[16]>(o));
      ptx::tmem_ld_wait();
#pragma unroll
      for (int x = 0; x < 16; ++x) o[x] = o[x] * part.down * unit;
#pragma unroll
      for (int x = 0; x < 16 && mine; x += 4)
        part_row<D>(P, slot, h, row)[(k + x) / 4 * kHalf] = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
    }
    read();
    if (mine) ml[slot * 2 * kHalf] = make_float2(m + part.up, l * part.down);
    if (!P.join_after && last_to_arrive(P, g, h, row == 0, last, bar, 128) && mine) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll 4
      for (int q = 0; q < g.parts; ++q)
        top = fmaxf(top, __ldcg(&ml[part_slot(g, q) * 2 * kHalf].x));
      const float ref = top == -INFINITY ? 0.f : top;
      for (int q = 0; q < g.parts; ++q) {
        const float2 v = __ldcg(&ml[part_slot(g, q) * 2 * kHalf]);
        sum += exp2_fast(v.x - ref) * v.y;
      }
      const RowWriter<D> joined(P, g.shared, t, head, true, top, sum);
#pragma unroll 1
      for (int k = 0; k < D; k += 16) {
        float o[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = 0.f;
#pragma unroll 2
        for (int q = 0; q < g.parts; ++q) {
          const float f = exp2_fast(__ldcg(&ml[part_slot(g, q) * 2 * kHalf].x) - ref);
          const float4* from = part_row<D>(P, part_slot(g, q), h, row) + k / 4 * kHalf;
#pragma unroll
          for (int x = 0; x < 16; x += 4) {
            const float4 z = __ldcg(from + x / 4 * kHalf);
            o[x] += f * z.x;
            o[x + 1] += f * z.y;
            o[x + 2] += f * z.z;
            o[x + 3] += f * z.w;
          }
        }
        joined.write16(k, o);
      }
    }
  } else {
    float o[D];
#pragma unroll
    for (int k = 0; k < D; k += 32)
      ptx::tmem_ld32(tm_o + k, *reinterpret_cast<uint32_t(*)[32]>(o + k));
    ptx::tmem_ld_wait();
    read();
    float2* ml = reinterpret_cast<float2*>(P.part_ml) + h * kHalf + row;
    if (mine) {
      float4* part = part_row<D>(P, slot, h, row);
#pragma unroll
      for (int k = 0; k < D; k += 4)
        part[(k / 4) * kHalf] = make_float4(o[k] * unit, o[k + 1] * unit, o[k + 2] * unit, o[k + 3] * unit);
      ml[slot * 2 * kHalf] = make_float2(m, l);
    }
    if (!P.join_after && last_to_arrive(P, g, h, row == 0, last, bar, 128) && mine) {
      // few parts: the last to arrive adds them up, in their order
      float top = -INFINITY, sum = 0.f;
#pragma unroll 4
      for (int q = 0; q < g.parts; ++q)
        top = fmaxf(top, __ldcg(&ml[part_slot(g, q) * 2 * kHalf].x));
#pragma unroll
      for (int k = 0; k < D; ++k) o[k] = 0.f;
#pragma unroll 1
      for (int q = 0; q < g.parts && top > -INFINITY; ++q) {
        const float2 v = __ldcg(&ml[part_slot(g, q) * 2 * kHalf]);
        const float f = exp2_fast(v.x - top);
        sum += f * v.y;
        const float4* from = part_row<D>(P, part_slot(g, q), h, row);
#pragma unroll
        for (int k = 0; k < D; k += 4) {
          const float4 z = __ldcg(from + (k / 4) * kHalf);
          o[k] += f * z.x;
          o[k + 1] += f * z.y;
          o[k + 2] += f * z.z;
          o[k + 3] += f * z.w;
        }
      }
      const RowWriter<D> joined(P, g.shared, t, head, true, top, sum);
#pragma unroll
      for (int k = 0; k < D; k += 16) joined.write16(k, o + k);
    }
  }
}

// The kernel that joins parts after an attention kernel (P.join_after), see k_attn_prefill.cu.
cudaError_t launch_attn_join(const AttnParams& P, cudaStream_t st);

}  // namespace lora
