// Rows of activations to int8 with one scale each, computed on the way: the
// residual's addition with an RMS norm (the x of a layer's q|k|v and gate|up
// products) and the gated activation (the x of its down product).
//
//   norm : h = x + r,  y = (h a) w,  a = f32(1 / sqrt(mean(h^2) + eps))
//   gated: y = act(gate) up
//   s = max|y| / 127 (1 for a row of zeros),  q = clip(rint(y / s), -127, 127)
//
// The steps from h or y on are single IEEE fp32 operations, so that codes are
// what the definition says, bit for bit; only the sum of squares is fp64 (squares
// of fp32 are exact there), so that its order does not show in a.
//
// One workgroup a row, which reads it once a pass.
#include "actq.h"
#include "kv4.h"

namespace sherry {
namespace {

// Sum over the workgroup (every thread gets it).
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d);
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < kActThreads / kWave; ++w) v += part[w];
  return v;
}

template <int DT>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
  if constexpr (DT == kActF32)
    gmem(static_cast<float*>(p))[i] = v;
  else
    gmem(static_cast<uint16_t*>(p))[i] = static_cast<uint16_t>(pack2<DT>(v, 0.0f));
}

template <int XDT, int RDT>
__global__ __launch_bounds__(kActThreads) void rms_norm_quant_kernel(NormQuantArgs a) {
  __shared__ double part[kActThreads / kWave];
  __shared__ float wmax[kActThreads / kWave];
  const int64_t row = blockIdx.x;
  auto value = [&](int64_t j) {
    const float x = act_value(a.x, XDT, row * a.ldx + j);
    if constexpr (RDT < 0) return x;
    return x + act_value(a.r, RDT, row * a.ldr + j);
  };
  double ss = 0.0;
  for (int64_t j = threadIdx.x; j < a.k; j += kActThreads) {
    const double h = value(j);
    ss = __builtin_fma(h, h, ss);
  }
  ss = block_sum(ss, part);
  const float inv = static_cast<float>(1.0 / __builtin_sqrt(ss / static_cast<double>(a.k) + static_cast<double>(a.eps)));
  float amax = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += kActThreads) amax = fmaxf(amax, fabsf(value(j) * inv * gmem(a.w)[j]));
  const float s = act_scale(block_max(amax, wmax));
  if (threadIdx.x == 0) gmem(a.scales)[row] = s;
  // (a thread reads r where it writes r_out, which may be the same memory)
  for (int64_t j = threadIdx.x; j < a.k; j += kActThreads) {
    const float h = value(j);
    gmem(a.q)[row * a.ldq + j] = act_code(h * inv * gmem(a.w)[j], s);
    if constexpr (RDT >= 0) put<RDT>(a.r_out, row * a.ldro + j, h);
  }
}

// g / (1 + exp(-z)): SiLU with z = g, and GELU with z = 2 sqrt(2/pi) (g + 0.044715 g^3),
// whose (1 + tanh(z/2)) / 2 this is without the cancellation.
__device__ __forceinline__ float activate(float g, int act) {
  const float z = act == kGateSilu ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g / (1.0f + expf(-z));
}

template <int DT>
__global__ __launch_bounds__(kActThreads) void gated_quant_kernel(GatedQuantArgs a) {
  __shared__ float wmax[kActThreads / kWave];
  const int64_t row = blockIdx.x;
  auto value = [&](int64_t j) {
    return activate(act_value(a.gate, DT, row * a.ldg + j), a.act) * act_value(a.up, DT, row * a.ldu + j);
  };
  float amax = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += kActThreads) amax = fmaxf(amax, fabsf(value(j)));
  const float s = act_scale(block_max(amax, wmax));
  if (threadIdx.x == 0) gmem(a.scales)[row] = s;
  for (int64_t j = threadIdx.x; j < a.k; j += kActThreads) gmem(a.q)[row * a.ldq + j] = act_code(value(j), s);
}

template <int XDT>
void launch_norm(const NormQuantArgs& a, int rdt, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.m)), block(kActThreads);
  if (!a.r)
    hipLaunchKernelGGL((rms_norm_quant_kernel<XDT, -1>), grid, block, 0, stream, a);
  else if (rdt == kActF32)
    hipLaunchKernelGGL((rms_norm_quant_kernel<XDT, kActF32>), grid, block, 0, stream, a);
  else if (rdt == kActF16)
    hipLaunchKernelGGL((rms_norm_quant_kernel<XDT, kActF16>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((rms_norm_quant_kernel<XDT, kActBf16>), grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_rms_norm_quant(const NormQuantArgs& a, int xdt, int rdt, hipStream_t stream) {
  if (xdt == kActF32)
    launch_norm<kActF32>(a, rdt, stream);
  else if (xdt == kActF16)
    launch_norm<kActF16>(a, rdt, stream);
  else
    launch_norm<kActBf16>(a, rdt, stream);
  return hipGetLastError();
}

hipError_t launch_gated_quant(const GatedQuantArgs& a, int dt, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.m)), block(kActThreads);
  if (dt == kActF32)
    hipLaunchKernelGGL((gated_quant_kernel<kActF32>), grid, block, 0, stream, a);
  else if (dt == kActF16)
    hipLaunchKernelGGL((gated_quant_kernel<kActF16>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((gated_quant_kernel<kActBf16>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace sherry
