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
// All heads of a lane rotate before the first is stored.  Stored one by one they take
// fewer registers where fp32 goes out (118 against 155 to 222, four waves a SIMD against
// two or three), but longer: 8192 tokens as above fp32 to fp32 72.0 us against 64.7, fp16
// to fp32 60.4 against 49.3, bf16 27.5 against 26.3; of 32 + 8 heads of 64 fp16 to fp32
// 37.9 against 27.3; 2048 tokens to fp32 17.3 against 18.3, one token the same.
#include "rope.h"

namespace sherry {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeHeads = 4;

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
  float x0[HPL][8], x1[HPL][8];
  int d0, d1;
  norm_rope<XDT, HPL>(a, t, tok, head, lane, has, x0, x1, d0, d1);
  if (!has) return;
#pragma unroll
  for (int h = 0; h < HPL; ++h) {
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
