// A head's norm and rotation in the lanes that hold it, shared by the rotation
// (rope.hip) and the cache append (kv4_append.hip).
#pragma once

#include "kv4.h"

namespace sherry {

__device__ __forceinline__ float sum_lanes_of(float v, int lph) {  // valid in every lane
  switch (lph) {
    case 16: return reduce_add_f32_last<16>(v);
    case 8: return reduce_add_f32_last<8>(v);
    case 4: return reduce_add_f32_last<4>(v);
    case 2: return reduce_add_f32_last<2>(v);
    default: return v;
  }
}

// Values of HPL heads from `head` on of token `tok`, normalised and rotated, in
// the lane's two runs of eight, d0 and d1 on.  A lane without values (has false)
// takes part in the reductions.  kAll: every lane has values, heads past the last
// being the last again, so that no load stands behind a branch; kFull: all of a head
// rotates, in half-split pairs.
template <int XDT, int HPL, bool kAll = false, bool kFull = false>
__device__ __forceinline__ void norm_rope(const RopeArgs& a, const RopeHeads& t, int64_t tok, int head, int lane, bool has,
                                          float (&x0)[HPL][8], float (&x1)[HPL][8], int& d0, int& d1) {
  const int lph = 1 << a.lph_shift;
  const bool rotates = kFull || 16 * lane < a.rot;
  // first values of the lane's two runs
  d0 = 16 * lane, d1 = d0 + 8;
  if (kFull || (rotates && !a.interleaved)) d0 = 8 * lane, d1 = d0 + a.rot / 2;
#pragma unroll
  for (int h = 0; h < HPL; ++h) {
    if constexpr (!kAll) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x0[h][j] = x1[h][j] = 0.0f;
    }
    if (kAll || (has && head + h < t.heads)) {
      const int64_t at = tok * t.x_st + (kAll ? min(head + h, t.heads - 1) : head + h) * t.x_sh;
      load8<XDT>(t.x, at + d0, x0[h]);
      load8<XDT>(t.x, at + d1, x1[h]);
    }
  }
  int64_t pos = 0;
  bool pos_ok = true;
  if ((kAll || has) && rotates) {
    pos = gmem(a.pos)[tok];
    pos_ok = pos >= 0 && pos < a.max_pos;
    if (!pos_ok) pos = 0;
  }
  // eight pairs: cos and sin 8 * lane .. + 7 in both styles
  float c[8], s[8];
  if ((kAll || has) && rotates) {
    const int64_t row = pos * (a.rot / 2) + 8 * lane;
    load8<kActF32>(a.cos, row, c);
    load8<kActF32>(a.sin, row, s);
    if (!pos_ok) {
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = __builtin_nanf("");
    }
  }
  if (t.w) {  // (every lane of a head takes the same way)
    float w0[8], w1[8];
    if constexpr (!kAll) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w0[j] = w1[j] = 0.0f;
    }
    if (kAll || has) {
      load8<kActF32>(t.w, d0, w0);
      load8<kActF32>(t.w, d1, w1);
    }
#pragma unroll
    for (int h = 0; h < HPL; ++h) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(x0[h][j], x0[h][j], __builtin_fmaf(x1[h][j], x1[h][j], ss));
      ss = sum_lanes_of(ss, lph);
      const float r = 1.0f / __builtin_sqrtf(ss / static_cast<float>(a.d) + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) x0[h][j] = x0[h][j] * r * w0[j], x1[h][j] = x1[h][j] * r * w1[j];
    }
  }
  if (!rotates) return;
#pragma unroll
  for (int h = 0; h < HPL; ++h) {
    float y0[8], y1[8];
    if (!kFull && a.interleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y0[2 * j] = x0[h][2 * j] * c[j] - x0[h][2 * j + 1] * s[j];
        y0[2 * j + 1] = x0[h][2 * j + 1] * c[j] + x0[h][2 * j] * s[j];
        y1[2 * j] = x1[h][2 * j] * c[4 + j] - x1[h][2 * j + 1] * s[4 + j];
        y1[2 * j + 1] = x1[h][2 * j + 1] * c[4 + j] + x1[h][2 * j] * s[4 + j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y0[j] = x0[h][j] * c[j] - x1[h][j] * s[j];
        y1[j] = x1[h][j] * c[j] + x0[h][j] * s[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x0[h][j] = y0[j], x1[h][j] = y1[j];
  }
}

}  // namespace sherry
