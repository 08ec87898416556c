// Rotation of 16-value units of a head by position: (a, b) -> (a c - b s, b c + a s) for
// pair i, c and s from the caller's table at the position of the pair's axis.  load_rot
// serves lora_kv_append, which rotates on the way to bf16; rotate_unit its 8-bit form,
// which has the rows' cosines and sines in shared memory.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace lora {

// cos and sin of a unit's eight pairs.
struct Rot {
  float c[8], s[8];
};

// Those of unit u for row t at position p.
__device__ __forceinline__ void load_rot(const AppendArgs& a, int T, int t, int p, int u, Rot& r) {
  auto pos_of = [&](int axis) {
    const int x = a.pos != nullptr ? a.pos[static_cast<int64_t>(axis) * T + t] : p;
    if (x >= 0 && x < a.n_pos) return x;
    flag_error(a.err, LORA_DEVERR_BAD_POS);
    return -1;
  };
  auto axis_of = [&](int pair) {
    int ax = 0;
#pragma unroll
    for (int i = 0; i < LORA_MAX_POS_AXES - 1; ++i) ax += pair >= a.axis_end[i] ? 1 : 0;
    return ax < a.n_axes ? ax : a.n_axes - 1;
  };
  const int ax = axis_of(8 * u);
  if (ax == axis_of(8 * u + 7)) {
    const int x = pos_of(ax);
    if (x >= 0) {
      const float* row = a.cos_sin + static_cast<int64_t>(x) * a.rot_dim + 8 * u;
      load8(row, r.c);
      load8(row + a.rot_dim / 2, r.s);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) r.c[j] = 1.f, r.s[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int x = pos_of(axis_of(8 * u + j));
      const float* row = a.cos_sin + static_cast<int64_t>(x < 0 ? 0 : x) * a.rot_dim + 8 * u + j;
      r.c[j] = x < 0 ? 1.f : row[0];
      r.s[j] = x < 0 ? 0.f : row[a.rot_dim / 2];
    }
  }
}

// A unit's two vectors of eight, x[0 .. 8) and x[8 .. 16): the pairs are (x[j], x[8 + j]),
// or neighbours with kInter.
template <bool kInter>
__device__ __forceinline__ void rotate_unit(float (&x)[16], const Rot& r) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int ia = kInter ? 2 * j : j, ib = kInter ? 2 * j + 1 : 8 + j;
    const float a = x[ia], b = x[ib];
    x[ia] = a * r.c[j] - b * r.s[j];
    x[ib] = b * r.c[j] + a * r.s[j];
  }
}

}  // namespace lora
