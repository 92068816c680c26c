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
// most 16 lanes.  Bound: HBM (each value is read and written once).
#include "kv4.h"

namespace sherry {
namespace {

constexpr int kRopeThreads = 256;

template <int W>
__device__ __forceinline__ float sum_lanes(float v) {  // valid in every lane for W <= 16
  return reduce_add_f32_last<W>(v);
}

__device__ __forceinline__ float sum_lanes_of(float v, int lph) {
  switch (lph) {
    case 16: return sum_lanes<16>(v);
    case 8: return sum_lanes<8>(v);
    case 4: return sum_lanes<4>(v);
    case 2: return sum_lanes<2>(v);
    default: return v;
  }
}

template <int XDT, int YDT>
__global__ __launch_bounds__(kRopeThreads) void qk_norm_rope_kernel(RopeArgs a) {
  const int lph = 1 << a.lph_shift;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x) >> a.lph_shift;
  const int lane = threadIdx.x & (lph - 1);
  const int heads = a.q.heads + a.k.heads;
  const int64_t tok = unit / heads;
  const bool live = tok < a.n;  // whole heads: every lane of a reduction agrees
  const int h = live ? static_cast<int>(unit - tok * heads) : 0;
  const RopeHeads& t = h < a.q.heads ? a.q : a.k;
  const int head = h < a.q.heads ? h : h - a.q.heads;
  const bool has = live && 16 * lane < a.d;
  const bool rotates = 16 * lane < a.rot;
  // first values of the lane's two runs
  int d0 = 16 * lane, d1 = d0 + 8;
  if (rotates && !a.interleaved) d0 = 8 * lane, d1 = d0 + a.rot / 2;
  float x0[8], x1[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x0[j] = x1[j] = 0.0f;
  if (has) {
    const int64_t at = tok * t.x_st + head * t.x_sh;
    load8<XDT>(t.x, at + d0, x0);
    load8<XDT>(t.x, at + d1, x1);
  }
  int64_t pos = 0;
  bool pos_ok = true;
  if (has && rotates) {
    pos = gmem(a.pos)[tok];
    pos_ok = pos >= 0 && pos < a.max_pos;
    if (!pos_ok) pos = 0;
  }
  if (t.w) {
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(x0[j], x0[j], __builtin_fmaf(x1[j], x1[j], ss));
    ss = sum_lanes_of(ss, lph);
    const float r = 1.0f / __builtin_sqrtf(ss / static_cast<float>(a.d) + a.eps);
    if (has) {
      float w0[8], w1[8];
      load8<kActF32>(t.w, d0, w0);
      load8<kActF32>(t.w, d1, w1);
#pragma unroll
      for (int j = 0; j < 8; ++j) x0[j] = x0[j] * r * w0[j], x1[j] = x1[j] * r * w1[j];
    }
  }
  if (!has) return;
  if (rotates) {
    // eight pairs: cos and sin 8 * lane .. + 7 in both styles
    float c[8], s[8];
    const int64_t row = pos * (a.rot / 2) + 8 * lane;
    load8<kActF32>(a.cos, row, c);
    load8<kActF32>(a.sin, row, s);
    if (!pos_ok) {
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = __builtin_nanf("");
    }
    if (a.interleaved) {
      float y0[8], y1[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y0[2 * j] = x0[2 * j] * c[j] - x0[2 * j + 1] * s[j];
        y0[2 * j + 1] = x0[2 * j + 1] * c[j] + x0[2 * j] * s[j];
        y1[2 * j] = x1[2 * j] * c[4 + j] - x1[2 * j + 1] * s[4 + j];
        y1[2 * j + 1] = x1[2 * j + 1] * c[4 + j] + x1[2 * j] * s[4 + j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x0[j] = y0[j], x1[j] = y1[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = x0[j], v = x1[j];
        x0[j] = u * c[j] - v * s[j];
        x1[j] = v * c[j] + u * s[j];
      }
    }
  }
  const int64_t to = tok * t.y_st + head * t.y_sh;
  store8<YDT>(t.y, to + d0, x0);
  store8<YDT>(t.y, to + d1, x1);
}

template <int XDT>
void launch_x(const RopeArgs& a, int ydt, dim3 grid, hipStream_t stream) {
  if (ydt == kActF32)
    hipLaunchKernelGGL((qk_norm_rope_kernel<XDT, kActF32>), grid, dim3(kRopeThreads), 0, stream, a);
  else if (ydt == kActF16)
    hipLaunchKernelGGL((qk_norm_rope_kernel<XDT, kActF16>), grid, dim3(kRopeThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<XDT, kActBf16>), grid, dim3(kRopeThreads), 0, stream, a);
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& a, int xdt, int ydt, hipStream_t stream) {
  const int64_t lanes = a.n * (a.q.heads + a.k.heads) << a.lph_shift;
  const dim3 grid(static_cast<unsigned>((lanes + kRopeThreads - 1) / kRopeThreads));
  if (xdt == kActF32)
    launch_x<kActF32>(a, ydt, grid, stream);
  else if (xdt == kActF16)
    launch_x<kActF16>(a, ydt, grid, stream);
  else
    launch_x<kActBf16>(a, ydt, grid, stream);
  return hipGetLastError();
}

}  // namespace sherry
