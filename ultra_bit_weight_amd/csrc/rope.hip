// RMS norms of query and key heads and the position rotation, in one pass over
// the fused projection's output (the step between a decoder layer's q|k|v
// product and its attention).
//
//   n = x * rsqrt(mean(x^2) + eps) * w        (skipped without w)
//   (a, b) -> (a cos - b sin, b cos + a sin)  for the pairs of the first rot
//                                             values; the others pass through
// All in fp32 with one rounding at the store.
//
// A head takes ceil(D / 16) lanes (rounded up to a power of two); each lane
// holds two runs of eight values, chosen so that every pair lies in one lane:
// half-split pairs (i, i + rot/2) as the two runs, neighbouring pairs inside a
// run.  So the rotation needs no exchange, and the norm one reduction over at
// most 16 lanes.  A lane takes the same runs of HPL heads, whose loads go out
// together and share the token's cosines and sines and the norm's weights: 4
// heads a lane where that still leaves the chip full, else 1 (a decode step is
// one wave's latency).
// Bound: HBM (each value is read and written once): 8192 tokens of 24 + 8 heads
// of 128 with norms in 25.5 us, 5.4 TB/s, the rate of a large copy.
#include "kv4.h"

namespace sherry {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeHeads = 4;

__device__ __forceinline__ float sum_lanes_of(float v, int lph) {  // valid in every lane
  switch (lph) {
    case 16: return reduce_add_f32_last<16>(v);
    case 8: return reduce_add_f32_last<8>(v);
    case 4: return reduce_add_f32_last<4>(v);
    case 2: return reduce_add_f32_last<2>(v);
    default: return v;
  }
}

template <int XDT, int YDT, int HPL, bool kStream>
__global__ __launch_bounds__(kRopeThreads) void qk_norm_rope_kernel(RopeArgs a) {
  const int lph = 1 << a.lph_shift;
  const uint32_t unit = (blockIdx.x * static_cast<uint32_t>(kRopeThreads) + threadIdx.x) >> a.lph_shift;
  const int lane = threadIdx.x & (lph - 1);
  const uint32_t q_sets = (a.q.heads + HPL - 1) / HPL, sets = q_sets + (a.k.heads + HPL - 1) / HPL;
  const uint32_t tok32 = unit / sets, set = unit - tok32 * sets;
  const int64_t tok = tok32;
  const RopeHeads& t = set < q_sets ? a.q : a.k;
  const int head = static_cast<int>((set < q_sets ? set : set - q_sets) * HPL);
  const bool has = tok < a.n && 16 * lane < a.d;
  const bool rotates = 16 * lane < a.rot;
  // first values of the lane's two runs
  int d0 = 16 * lane, d1 = d0 + 8;
  if (rotates && !a.interleaved) d0 = 8 * lane, d1 = d0 + a.rot / 2;
  float x0[HPL][8], x1[HPL][8];
#pragma unroll
  for (int h = 0; h < HPL; ++h) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x0[h][j] = x1[h][j] = 0.0f;
    if (has && head + h < t.heads) {
      const int64_t at = tok * t.x_st + (head + h) * t.x_sh;
      load8<XDT>(t.x, at + d0, x0[h]);
      load8<XDT>(t.x, at + d1, x1[h]);
    }
  }
  int64_t pos = 0;
  bool pos_ok = true;
  if (has && rotates) {
    pos = gmem(a.pos)[tok];
    pos_ok = pos >= 0 && pos < a.max_pos;
    if (!pos_ok) pos = 0;
  }
  // eight pairs: cos and sin 8 * lane .. + 7 in both styles
  float c[8], s[8];
  if (has && rotates) {
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
#pragma unroll
    for (int j = 0; j < 8; ++j) w0[j] = w1[j] = 0.0f;
    if (has) {
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
  if (!has) return;
#pragma unroll
  for (int h = 0; h < HPL; ++h) {
    if (rotates) {
      float y0[8], y1[8];
      if (a.interleaved) {
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
    if (head + h < t.heads) {
      const int64_t to = tok * t.y_st + (head + h) * t.y_sh;
      store8<YDT, kStream>(t.y, to + d0, x0[h]);
      store8<YDT, kStream>(t.y, to + d1, x1[h]);
    }
  }
}

template <int XDT, int YDT>
void launch_xy(const RopeArgs& a, hipStream_t stream) {
  auto grid = [&](int hpl) {
    const int64_t sets = (a.q.heads + hpl - 1) / hpl + (a.k.heads + hpl - 1) / hpl;
    return static_cast<unsigned>(((a.n * sets << a.lph_shift) + kRopeThreads - 1) / kRopeThreads);
  };
  const dim3 block(kRopeThreads);
  const unsigned many = grid(kRopeHeads);
  if (a.n * (a.q.heads + a.k.heads) * a.d * act_bytes(YDT) > kStreamBytes)
    hipLaunchKernelGGL((qk_norm_rope_kernel<XDT, YDT, kRopeHeads, true>), dim3(many), block, 0, stream, a);
  else if (many >= 1024)
    hipLaunchKernelGGL((qk_norm_rope_kernel<XDT, YDT, kRopeHeads, false>), dim3(many), block, 0, stream, a);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<XDT, YDT, 1, false>), dim3(grid(1)), block, 0, stream, a);
}

template <int XDT>
void launch_x(const RopeArgs& a, int ydt, hipStream_t stream) {
  if (ydt == kActF32)
    launch_xy<XDT, kActF32>(a, stream);
  else if (ydt == kActF16)
    launch_xy<XDT, kActF16>(a, stream);
  else
    launch_xy<XDT, kActBf16>(a, stream);
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& a, int xdt, int ydt, hipStream_t stream) {
  if (xdt == kActF32)
    launch_x<kActF32>(a, ydt, stream);
  else if (xdt == kActF16)
    launch_x<kActF16>(a, ydt, stream);
  else
    launch_x<kActBf16>(a, ydt, stream);
  return hipGetLastError();
}

}  // namespace sherry
