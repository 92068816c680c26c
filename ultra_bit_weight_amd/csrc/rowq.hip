// Rows of activations to int8 with one scale each, computed on the way: the
// residual's addition with an RMS norm (the x of a layer's q|k|v and gate|up
// products) and the gated activation (the x of its down product).
//
//   norm : h = x + r,  y = (h a) w,  a = f32(1 / sqrt(mean(h^2) + eps))
//   gated: y = act(gate) up
//   s = max|y| / 127 (1 for a row of zeros),  q = clip(rint(y / s), -127, 127)
//
// The norm's steps outside a are single IEEE fp32 operations, so that codes are
// what the definition says, bit for bit; only the sum of squares is fp64 (squares
// of fp32 are exact there), so that its order does not show in a.
//
// Bound by HBM: a row is read once and stays in its threads' registers through
// both reductions.  T threads take a row, V runs of eight values each.  8192 rows of
// 4096 in 16 bits with their residual 44-46 us, 5.2 TB/s, the rate of a large copy;
// 8192 rows of gate and up, 8192 each, 60 us, 5.6 TB/s; one row 2.75 and 3.15 us, a
// launch and one load-reduce-store.
#include <type_traits>

#include "actq.h"
#include "kv4.h"

namespace sherry {
namespace {

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xF, false));
  const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xF, false));
  return v + __builtin_bit_cast(double, lo | hi << 32);
}

// Reductions over a row's T threads (whole waves); every thread gets the result.
template <int T>
struct RowTeam {
  static constexpr int kWaves = T / kWave;
  __device__ static __forceinline__ double sum(double v, double* part) {
    v = dpp_add_f64<0xB1, 0xF>(v);   // quad_perm [1,0,3,2]
    v = dpp_add_f64<0x4E, 0xF>(v);   // quad_perm [2,3,0,1]
    v = dpp_add_f64<0x141, 0xF>(v);  // row_half_mirror
    v = dpp_add_f64<0x140, 0xF>(v);  // row_mirror
    v = dpp_add_f64<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
    v = dpp_add_f64<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b), kWave - 1));
    const uint64_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b >> 32), kWave - 1));
    v = __builtin_bit_cast(double, lo | hi << 32);
    if constexpr (kWaves > 1) {
      if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
      __syncthreads();
      v = part[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += part[w];
    }
    return v;
  }
  __device__ static __forceinline__ float max(float v, float* part) {
    v = dpp_max<0xB1, 0xF>(v);
    v = dpp_max<0x4E, 0xF>(v);
    v = dpp_max<0x141, 0xF>(v);
    v = dpp_max<0x140, 0xF>(v);
    v = dpp_max<0x142, 0xA>(v);
    v = dpp_max<0x143, 0xC>(v);
    v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), kWave - 1));
    if constexpr (kWaves > 1) {
      if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
      __syncthreads();
      v = part[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v = fmaxf(v, part[w]);
    }
    return v;
  }
};

// A vector at addresses of A bytes' alignment.
template <class W, int A>
struct __attribute__((packed, aligned(A))) Vec {
  W v;
};

// Eight values as they lie, B bytes each, aligned as 16 bytes or (kLoose) as one value.
template <int B>
struct Raw8 {
  u32x4_t w[B / 2];
  template <bool kLoose>
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    typedef Vec<u32x4_t, kLoose ? B : 16> vec_t;
    const SHERRY_GLOBAL vec_t* at = gmem(reinterpret_cast<const vec_t*>(static_cast<const char*>(p) + i * B));
#pragma unroll
    for (int j = 0; j < B / 2; ++j) w[j] = at[j].v;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < B / 2; ++j) w[j] = u32x4_t{0, 0, 0, 0};
  }
};
template <>
struct Raw8<0> {
  template <bool kLoose>
  __device__ __forceinline__ void load(const void*, int64_t) {}
  __device__ __forceinline__ void clear() {}
};

// to fp32; which of the 16-bit types it is, is the same for all of a launch
template <int B, int V>
__device__ __forceinline__ void widen(const Raw8<B> (&r)[V], int dt, float (&v)[V][8]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (B == 4)
          v[i][j] = __uint_as_float(r[i].w[j >> 2][j & 3]);
        else
          v[i][j] = f((r[i].w[0][j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
      }
  };
  if (B == 4 || dt == kActF16)
    each([](uint32_t h) { return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h))); });
  else
    each([](uint32_t h) { return __uint_as_float(h << 16); });
}

// A row's codes from its values: y / s by a product with 1 / s, which is within
// 127 * 3 * 2^-24 < 2^-15 of the quotient, so that both round to the same integer
// unless one comes that near to a half; then, and where 1 / s or the product would
// leave the normal numbers, the quotients themselves.  Adding 1.5 * 2^23 rounds
// half to even and leaves the integer in the low byte; no |y / s| passes 127 by
// more than a rounding.
template <bool kLoose, int V>
__device__ __forceinline__ void put_codes(const float (&y)[V][8], float s, int8_t* q, int k, int step) {
  const float inv = 1.0f / s;
  constexpr float kMagic = 12582912.0f;
  u32x2_t c[V];
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float t = y[i][4 * h + j] * inv, r = t + kMagic;
        far = fmaxf(far, fabsf(t - (r - kMagic)));
        b[j] = __float_as_uint(r);
      }
      c[i][h] = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u) | __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
    }
  if (__builtin_expect(__any(far > 0.5f - 0x1p-15f) || s < 0x1p-100f || s > 0x1p100f, 0)) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w |= static_cast<uint32_t>(static_cast<uint8_t>(act_code(y[i][4 * h + j], s))) << (8 * j);
        c[i][h] = w;
      }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = i * step;
    if (at + (kLoose ? 7 : 0) < k)
      gmem(reinterpret_cast<Vec<u32x2_t, kLoose ? 1 : 8>*>(q + at))->v = c[i];
    else if (kLoose && at < k)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + 8 - k <= j) gmem(q + k - 8)[j] = static_cast<int8_t>(c[i][j >> 2] >> (8 * (j & 3)));
  }
}

// 1 / sqrt(mean + eps) within 2^-50: the hardware's estimate and two Newton steps (a
// third of the latency of an exact root and quotient, which every row waits for).
// Nothing at all under the root: the row is zeros, and so are its values.  Without eps a
// row below 2^-128 has a factor past fp32: the largest one, so that zeros stay zeros.
__device__ __forceinline__ float norm_factor(double ss, const NormQuantArgs& a) {
  const double x = __builtin_fma(ss, a.inv_k, static_cast<double>(a.eps));
  double y = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = __builtin_fma(__builtin_fma(-x * y, y, 1.0), 0.5 * y, y);
  return x > 0.0 ? fminf(static_cast<float>(y), 0x1.fffffep127f) : 0.0f;
}

template <int V>
__device__ __forceinline__ float top_of(const float (&y)[V][8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[i][j]));
  return m;
}

// Threads of a workgroup: one row's, or four rows of one wave each (which meet at no
// barrier).
constexpr int row_block(int t) { return t == kWave ? 4 * t : t; }

// kLoose: rows of any length from eight, at any address and stride.  The hardware takes
// vector loads and stores at any address; a row's last run, where fewer than eight
// values are left, is its last eight, of which those that the run before holds count
// as zeros and are not stored (so that it does not matter whether the run before has
// stored them, where r_out is r or x).  209 rows of 9213 values 5.2 us, 31 value by value;
// 8192 of 2049 34.6, 110; 8192 of gate and up, 8191 each, 66, 264 (8192 each, aligned,
// 60).
template <bool kLoose, int V>
__device__ __forceinline__ void drop_before(float (&h)[V][8], int c0, int step, int k) {
  if constexpr (kLoose)
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = c0 + i * step + 8 - k <= j ? h[i][j] : 0.0f;
}

template <int DT>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
  if constexpr (DT == kActF32)
    gmem(static_cast<float*>(p))[i] = v;
  else
    gmem(static_cast<uint16_t*>(p))[i] = static_cast<uint16_t>(pack2<DT>(v, 0.0f));
}

// eight values at any address
template <int DT>
__device__ __forceinline__ void put8(void* p, int64_t i, const float (&v)[8]) {
  constexpr int B = DT == kActF32 ? 4 : 2;
  SHERRY_GLOBAL Vec<u32x4_t, B>* to = gmem(reinterpret_cast<Vec<u32x4_t, B>*>(static_cast<char*>(p) + i * B));
#pragma unroll
  for (int h = 0; h < B / 2; ++h) {
    u32x4_t w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = B == 4 ? __float_as_uint(v[4 * h + j]) : pack2<DT>(v[2 * j], v[2 * j + 1]);
    to[h].v = w;
  }
}

template <int RB, bool kLoose, int V>
__device__ __forceinline__ void put_sum(const NormQuantArgs& a, int64_t row, int c0, int step, int rdt, const float (&h)[V][8]) {
  const int k = static_cast<int>(a.k);
  auto store = [&](auto dt) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = c0 + i * step;
      if constexpr (!kLoose) {
        if (c < k) store8<decltype(dt)::value>(a.r_out, row * a.ldro + c, h[i]);
      } else if (c + 8 <= k) {
        put8<decltype(dt)::value>(a.r_out, row * a.ldro + c, h[i]);
      } else if (c < k) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + 8 - k <= j) put<decltype(dt)::value>(a.r_out, row * a.ldro + k - 8 + j, h[i][j]);
      }
    }
  };
  if constexpr (RB == 4)
    store(std::integral_constant<int, kActF32>{});
  else if (rdt == kActF16)
    store(std::integral_constant<int, kActF16>{});
  else
    store(std::integral_constant<int, kActBf16>{});
}

template <int XB, int RB, bool kLoose, int T, int V>
__global__ __launch_bounds__(row_block(T)) void rms_norm_quant_rows(NormQuantArgs a, int xdt, int rdt) {
  __shared__ double part[T / kWave];
  __shared__ float wmax[T / kWave];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (row_block(T) / T) + threadIdx.x / T;
  if (row >= a.m) return;  // (whole waves, and only where a row is one)
  const int k = static_cast<int>(a.k), c0 = static_cast<int>(threadIdx.x % T) * 8;
  Raw8<XB> x[V];
  Raw8<RB> r[V];
  Raw8<4> w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = min(c0 + i * T * 8, k - 8);
    x[i].template load<kLoose>(a.x, row * a.ldx + c);
    r[i].template load<kLoose>(a.r, row * a.ldr + c);
    w[i].template load<kLoose>(a.w, c);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {  // (runs past the row's end loaded its last, so that no load stands behind a branch)
    if (c0 + i * T * 8 < k) continue;
    x[i].clear();
    r[i].clear();
  }
  float h[V][8];
  widen<XB, V>(x, xdt, h);
  if constexpr (RB > 0) {
    float g[V][8];
    widen<RB, V>(r, rdt, g);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += g[i][j];
    put_sum<RB, kLoose, V>(a, row, c0, T * 8, rdt, h);
  }
  drop_before<kLoose, V>(h, c0, T * 8, k);
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fma(static_cast<double>(h[i][j]), static_cast<double>(h[i][j]), ss);
  ss = RowTeam<T>::sum(ss, part);
  const float inv = norm_factor(ss, a);
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * inv * __uint_as_float(w[i].w[j >> 2][j & 3]);
  const float s = act_scale(RowTeam<T>::max(top_of<V>(h), wmax));
  if (c0 == 0) gmem(a.scales)[row] = s;
  put_codes<kLoose, V>(h, s, a.q + row * a.ldq + c0, k - c0, T * 8);
}

// g / (1 + exp(-z)): SiLU with z = g, and GELU with z = 2 sqrt(2/pi) (g + 0.044715 g^3),
// whose (1 + tanh(z/2)) / 2 this is without the cancellation.  The exponential is the
// hardware's, of one rounded product: its error grows with |z| where z < 0 (31 units in
// the last place at -85, 84 of GELU at z = -87; 1.5 for z > 0).  Such a value is e^z times
// an ordinary one, and codes keep seven bits of the row's largest.
__device__ __forceinline__ float activate(float g, int act) {
  const float z = act == kGateSilu ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}

// which activation it is, is the same for all of a launch
template <int V>
__device__ __forceinline__ void gate(float (&y)[V][8], const float (&v)[V][8], int act) {
  auto each = [&](int act) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] = activate(y[i][j], act) * v[i][j];
  };
  if (act == kGateSilu)
    each(kGateSilu);
  else
    each(kGateGeluTanh);
}

template <int XB, bool kLoose, int T, int V>
__global__ __launch_bounds__(row_block(T)) void gated_quant_rows(GatedQuantArgs a, int dt) {
  __shared__ float wmax[T / kWave];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (row_block(T) / T) + threadIdx.x / T;
  if (row >= a.m) return;
  const int k = static_cast<int>(a.k), c0 = static_cast<int>(threadIdx.x % T) * 8;
  Raw8<XB> g[V], u[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = min(c0 + i * T * 8, k - 8);
    g[i].template load<kLoose>(a.gate, row * a.ldg + c);
    u[i].template load<kLoose>(a.up, row * a.ldu + c);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (c0 + i * T * 8 < k) continue;
    g[i].clear();
    u[i].clear();
  }
  float y[V][8], v[V][8];
  widen<XB, V>(g, dt, y);
  widen<XB, V>(u, dt, v);
  gate<V>(y, v, a.act);
  drop_before<kLoose, V>(y, c0, T * 8, k);
  const float s = act_scale(RowTeam<T>::max(top_of<V>(y), wmax));
  if (c0 == 0) gmem(a.scales)[row] = s;
  put_codes<kLoose, V>(y, s, a.q + row * a.ldq + c0, k - c0, T * 8);
}

// ---- rows that no workgroup's registers hold: the same runs, read again for each pass
// (4096 rows of 40000 with an fp32 residual 525 us, 1460 where the passes went value by
// value; 2048 of gate and up, 53248 each, 145 us, 493) ----

constexpr int kLong = 1024;  // threads a row, of two runs at once

template <int XB, int RB>
__global__ __launch_bounds__(kLong) void rms_norm_quant_long(NormQuantArgs a, int xdt, int rdt) {
  __shared__ double part[kLong / kWave];
  __shared__ float wmax[kLong / kWave];
  constexpr int V = 2, kStep = kLong * 8;
  const int64_t row = blockIdx.x;
  const int k = static_cast<int>(a.k), first = static_cast<int>(threadIdx.x) * 8;
  auto values = [&](int c0, float (&h)[V][8]) {
    Raw8<XB> x[V];
    Raw8<RB> r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = min(c0 + i * kStep, k - 8);
      x[i].template load<true>(a.x, row * a.ldx + c);
      r[i].template load<true>(a.r, row * a.ldr + c);
    }
    widen<XB, V>(x, xdt, h);
    if constexpr (RB > 0) {
      float g[V][8];
      widen<RB, V>(r, rdt, g);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += g[i][j];
    }
    drop_before<true, V>(h, c0, kStep, k);
  };
  auto scaled = [&](int c0, float (&h)[V][8], float inv) {
    Raw8<4> w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i].template load<true>(a.w, min(c0 + i * kStep, k - 8));
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * inv * __uint_as_float(w[i].w[j >> 2][j & 3]);
  };
  float h[V][8];
  double ss = 0.0;
  for (int c0 = first; c0 < k; c0 += V * kStep) {
    values(c0, h);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __builtin_fma(static_cast<double>(h[i][j]), static_cast<double>(h[i][j]), ss);
  }
  ss = RowTeam<kLong>::sum(ss, part);
  const float inv = norm_factor(ss, a);
  float amax = 0.0f;
  for (int c0 = first; c0 < k; c0 += V * kStep) {
    values(c0, h);
    scaled(c0, h, inv);
    amax = fmaxf(amax, top_of<V>(h));
  }
  const float s = act_scale(RowTeam<kLong>::max(amax, wmax));
  if (threadIdx.x == 0) gmem(a.scales)[row] = s;
  // (a thread reads the values of r and x that count for it where it writes r_out, which
  // may be the same memory)
  for (int c0 = first; c0 < k; c0 += V * kStep) {
    values(c0, h);
    if constexpr (RB > 0) put_sum<RB, true, V>(a, row, c0, kStep, rdt, h);
    scaled(c0, h, inv);
    put_codes<true, V>(h, s, a.q + row * a.ldq + c0, k - c0, kStep);
  }
}

template <int XB>
__global__ __launch_bounds__(kLong) void gated_quant_long(GatedQuantArgs a, int dt) {
  __shared__ float wmax[kLong / kWave];
  constexpr int V = 2, kStep = kLong * 8;
  const int64_t row = blockIdx.x;
  const int k = static_cast<int>(a.k), first = static_cast<int>(threadIdx.x) * 8;
  auto values = [&](int c0, float (&y)[V][8]) {
    Raw8<XB> g[V], u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = min(c0 + i * kStep, k - 8);
      g[i].template load<true>(a.gate, row * a.ldg + c);
      u[i].template load<true>(a.up, row * a.ldu + c);
    }
    float v[V][8];
    widen<XB, V>(g, dt, y);
    widen<XB, V>(u, dt, v);
    gate<V>(y, v, a.act);
    drop_before<true, V>(y, c0, kStep, k);
  };
  float y[V][8], amax = 0.0f;
  for (int c0 = first; c0 < k; c0 += V * kStep) {
    values(c0, y);
    amax = fmaxf(amax, top_of<V>(y));
  }
  const float s = act_scale(RowTeam<kLong>::max(amax, wmax));
  if (threadIdx.x == 0) gmem(a.scales)[row] = s;
  for (int c0 = first; c0 < k; c0 += V * kStep) {
    values(c0, y);
    put_codes<true, V>(y, s, a.q + row * a.ldq + c0, k - c0, kStep);
  }
}

// ---- rows of fewer than eight values: a wave a row, a value a lane ----

__global__ __launch_bounds__(row_block(kWave)) void rms_norm_quant_short(NormQuantArgs a, int xdt, int rdt) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (row_block(kWave) / kWave) + threadIdx.x / kWave;
  if (row >= a.m) return;
  const int j = static_cast<int>(threadIdx.x & (kWave - 1));
  const bool in = j < a.k;
  float h = 0.0f, w = 0.0f;
  if (in) {
    h = act_value(a.x, xdt, row * a.ldx + j);
    w = gmem(a.w)[j];
    if (a.r) h += act_value(a.r, rdt, row * a.ldr + j);
  }
  const double ss = RowTeam<kWave>::sum(static_cast<double>(h) * h, nullptr);
  const float y = h * norm_factor(ss, a) * w;
  const float s = act_scale(RowTeam<kWave>::max(fabsf(y), nullptr));
  if (j == 0) gmem(a.scales)[row] = s;
  if (!in) return;
  gmem(a.q)[row * a.ldq + j] = act_code(y, s);
  if (!a.r) return;
  if (rdt == kActF32)
    put<kActF32>(a.r_out, row * a.ldro + j, h);
  else if (rdt == kActF16)
    put<kActF16>(a.r_out, row * a.ldro + j, h);
  else
    put<kActBf16>(a.r_out, row * a.ldro + j, h);
}

__global__ __launch_bounds__(row_block(kWave)) void gated_quant_short(GatedQuantArgs a, int dt) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (row_block(kWave) / kWave) + threadIdx.x / kWave;
  if (row >= a.m) return;
  const int j = static_cast<int>(threadIdx.x & (kWave - 1));
  const bool in = j < a.k;
  float y = 0.0f;
  if (in) y = activate(act_value(a.gate, dt, row * a.ldg + j), a.act) * act_value(a.up, dt, row * a.ldu + j);
  const float s = act_scale(RowTeam<kWave>::max(fabsf(y), nullptr));
  if (j == 0) gmem(a.scales)[row] = s;
  if (in) gmem(a.q)[row * a.ldq + j] = act_code(y, s);
}

// ---- which threads a row gets ----

// Rows of whole runs of eight whose every run is aligned.
bool row_runs(const void* p, int64_t ld, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % (8 * bytes < 16 ? 8 * bytes : 16) == 0 && ld % 8 == 0;
}

// Calls f(T, V) as constants: as many threads as the row has runs of eight, so that
// what a thread waits for is one load, one reduction, one store; a long row gives
// them two or four.  Measured (us, 16-bit types; norm / gated, with 64 threads a row
// up to 4096 values and 256 beyond, as here, with two runs a thread):
//   8192 rows of 2048: 29.4 / 16.9, 24.9 / 15.4, 25.2 / 15.7
//   8192 of 4096:      58.8 / 36.7, 45.5 / 32.1, 45.2 / 32.6
//   8192 of 8192:      90.6 / 64.5, 85.3 / 61.0 (the norm with two runs, whose
//                      registers leave room for one row more a CU; 93.5 with one),
//                      85.3 / 63.5
//   4096 of 16384:     105 / 65.5, 88.3 / 61.0
// The threads go up by a half and a third, since waves without values take a row's
// place on a CU all the same: by doublings alone 8192 rows of 1280 took 17.0 / 14.1 (now
// 14.7 / 12.0), of 2560 34.5 / 25.8 (30.7 / 23.7), 4096 of gate and up, 18944 each,
// 108 (91).
template <bool kNorm, class F>
bool row_shape(int64_t k, F f) {
  auto go = [&](auto t, auto v) {
    f(t, v);
    return true;
  };
#define SHERRY_ROW(T, V) \
  if (k <= (T) * (V) * 8) return go(std::integral_constant<int, T>{}, std::integral_constant<int, V>{})
  SHERRY_ROW(64, 1);
  SHERRY_ROW(128, 1);
  SHERRY_ROW(192, 1);
  SHERRY_ROW(256, 1);
  SHERRY_ROW(384, 1);
  SHERRY_ROW(512, 1);
  if constexpr (kNorm) {
    SHERRY_ROW(512, 2);
  } else {
    SHERRY_ROW(768, 1);
    SHERRY_ROW(1024, 1);
  }
  SHERRY_ROW(768, 2);
  SHERRY_ROW(1024, 2);
  SHERRY_ROW(768, 4);
  SHERRY_ROW(1024, 4);
#undef SHERRY_ROW
  return false;
}

template <int T>
dim3 row_grid(int64_t m) {
  constexpr int rows = row_block(T) / T;
  return dim3(static_cast<unsigned>((m + rows - 1) / rows));
}

template <int XB, int RB, bool kLoose>
void launch_norm_rows(const NormQuantArgs& a, int xdt, int rdt, hipStream_t stream) {
  const bool done = row_shape<true>(a.k, [&](auto t, auto v) {
    constexpr int T = decltype(t)::value, V = decltype(v)::value;
    hipLaunchKernelGGL((rms_norm_quant_rows<XB, RB, kLoose, T, V>), row_grid<T>(a.m), dim3(row_block(T)), 0, stream, a, xdt,
                       rdt);
  });
  if (!done) hipLaunchKernelGGL((rms_norm_quant_long<XB, RB>), dim3(static_cast<unsigned>(a.m)), dim3(kLong), 0, stream, a, xdt, rdt);
}

template <bool kLoose>
void launch_norm(const NormQuantArgs& a, int xdt, int rdt, int64_t xb, int64_t rb, hipStream_t stream) {
  if (xb == 2)
    return rb == 0 ? launch_norm_rows<2, 0, kLoose>(a, xdt, rdt, stream)
           : rb == 2 ? launch_norm_rows<2, 2, kLoose>(a, xdt, rdt, stream) : launch_norm_rows<2, 4, kLoose>(a, xdt, rdt, stream);
  return rb == 0 ? launch_norm_rows<4, 0, kLoose>(a, xdt, rdt, stream)
         : rb == 2 ? launch_norm_rows<4, 2, kLoose>(a, xdt, rdt, stream) : launch_norm_rows<4, 4, kLoose>(a, xdt, rdt, stream);
}

template <int XB, bool kLoose>
void launch_gated(const GatedQuantArgs& a, int dt, hipStream_t stream) {
  const bool done = row_shape<false>(a.k, [&](auto t, auto v) {
    constexpr int T = decltype(t)::value, V = decltype(v)::value;
    hipLaunchKernelGGL((gated_quant_rows<XB, kLoose, T, V>), row_grid<T>(a.m), dim3(row_block(T)), 0, stream, a, dt);
  });
  if (!done) hipLaunchKernelGGL((gated_quant_long<XB>), dim3(static_cast<unsigned>(a.m)), dim3(kLong), 0, stream, a, dt);
}

}  // namespace

hipError_t launch_rms_norm_quant(const NormQuantArgs& a, int xdt, int rdt, hipStream_t stream) {
  const int64_t xb = act_bytes(xdt), rb = a.r ? act_bytes(rdt) : 0;
  const bool runs = a.k % 8 == 0 && row_runs(a.x, a.ldx, xb) && row_runs(a.q, a.ldq, 1) && row_runs(a.w, 8, 4) &&
                    (!a.r || (row_runs(a.r, a.ldr, rb) && row_runs(a.r_out, a.ldro, rb)));
  if (a.k < 8)
    hipLaunchKernelGGL(rms_norm_quant_short, row_grid<kWave>(a.m), dim3(row_block(kWave)), 0, stream, a, xdt, rdt);
  else if (runs)
    launch_norm<false>(a, xdt, rdt, xb, rb, stream);
  else
    launch_norm<true>(a, xdt, rdt, xb, rb, stream);
  return hipGetLastError();
}

hipError_t launch_gated_quant(const GatedQuantArgs& a, int dt, hipStream_t stream) {
  const int64_t b = act_bytes(dt);
  const bool runs = a.k % 8 == 0 && row_runs(a.gate, a.ldg, b) && row_runs(a.up, a.ldu, b) && row_runs(a.q, a.ldq, 1);
  if (a.k < 8)
    hipLaunchKernelGGL(gated_quant_short, row_grid<kWave>(a.m), dim3(row_block(kWave)), 0, stream, a, dt);
  else if (b == 2)
    runs ? launch_gated<2, false>(a, dt, stream) : launch_gated<2, true>(a, dt, stream);
  else
    runs ? launch_gated<4, false>(a, dt, stream) : launch_gated<4, true>(a, dt, stream);
  return hipGetLastError();
}

}  // namespace sherry
