// Writing keys and values into the 4-bit cache, and reading them back.
//
// For 64 consecutive values x of one token and head:
//   z = f16(min x), s = f16((max x - min x) / 15), clamped to +-65504
//   c = clip(rint((x - z) / s), 0, 15), 0 where s = 0     (IEEE fp32 steps)
//   value = z + s c                                       (one fp32 rounding)
//
// Eight lanes take a group, eight values each: the extremes are one three-step
// DPP reduction, and a lane's codes are whole nibbles of the layout's dwords.
// Bound: HBM (K and V are read once, a quarter of them written).
#include "kv4.h"

namespace sherry {
namespace {

constexpr int kKv4Threads = 256;

__device__ __forceinline__ float f16_clamped(float v, _Float16* h) {
  *h = static_cast<_Float16>(fminf(fmaxf(v, -65504.0f), 65504.0f));
  return static_cast<float>(*h);
}

template <int CTRL>
__device__ __forceinline__ float dpp_of(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}

// Codes of the lane's eight values; the eight lanes of a group share s and z.
__device__ __forceinline__ void quantise8(const float (&v)[8], uint32_t (&c)[8], _Float16* s16, _Float16* z16) {
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) lo = fminf(lo, v[j]), hi = fmaxf(hi, v[j]);
  lo = fminf(lo, dpp_of<0xB1>(lo)), hi = fmaxf(hi, dpp_of<0xB1>(hi));    // quad_perm [1,0,3,2]
  lo = fminf(lo, dpp_of<0x4E>(lo)), hi = fmaxf(hi, dpp_of<0x4E>(hi));    // quad_perm [2,3,0,1]
  lo = fminf(lo, dpp_of<0x141>(lo)), hi = fmaxf(hi, dpp_of<0x141>(hi));  // row_half_mirror
  const float z = f16_clamped(lo, z16);
  const float s = f16_clamped(__fdiv_rn(hi - lo, 15.0f), s16);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float r = s > 0.0f ? __builtin_rintf(__fdiv_rn(v[j] - z, s)) : 0.0f;
    c[j] = static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(r, 0.0f), 15.0f)));
  }
}

template <int D, int DT>
__global__ __launch_bounds__(kKv4Threads) void kv4_write_kernel(Kv4Geom g, Kv4Rows r) {
  using L = Kv4Layout<D>;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kKv4Threads + threadIdx.x) >> 3;
  const int l8 = threadIdx.x & 7;
  const int gr = static_cast<int>(unit % L::kGroups);
  const int64_t th = unit / L::kGroups;
  const int64_t tok = th / g.n_kv_heads;
  if (tok >= r.n) return;  // whole groups of eight lanes
  const int head = static_cast<int>(th - tok * g.n_kv_heads);
  const int64_t slot = gmem(r.slots)[tok];
  const int64_t page = slot >> g.page_shift;
  if (slot < 0 || page >= g.n_pages) return;
  const int in_page = static_cast<int>(slot & ((1 << g.page_shift) - 1));
  const int t = in_page & (kKv4Block - 1);
  uint8_t* blk = g.data + kv4_block_off<D>(g, page, head, in_page / kKv4Block);
  float v[8];
  uint32_t c[8];
  _Float16 s16, z16;
  // K: low nibbles come from lanes 0-3 of the group, high ones from 4-7
  load8<DT>(r.k, tok * r.k_st + head * r.k_sh + gr * kKv4Group + 8 * l8, v);
  quantise8(v, c, &s16, &z16);
  u32x2_t w = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j >> 2] |= c[j] << (8 * kv4_byte(j & 3));
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] |= static_cast<uint32_t>(__shfl_xor(static_cast<int>(w[i]), 4)) << 4;
  if (l8 < 4) *gmem(reinterpret_cast<u32x2_t*>(blk + L::k_off(t, gr, l8))) = w;
  if (l8 == 0) {
    *gmem(reinterpret_cast<_Float16*>(blk + L::p_off(t, gr, 0))) = s16;
    *gmem(reinterpret_cast<_Float16*>(blk + L::p_off(t, gr, 1))) = z16;
  }
  // V: a byte holds two values 16 apart, so lanes two apart share bytes; each
  // of the two stores four of their eight
  load8<DT>(r.v, tok * r.v_st + head * r.v_sh + gr * kKv4Group + 8 * l8, v);
  quantise8(v, c, &s16, &z16);
  const int high = (l8 >> 1) & 1;
  const int q = 2 * gr + (l8 >> 2);
  const int d16 = (l8 & 1) * 8 + high * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t mine = high ? c[4 + j] : c[j];
    const uint32_t theirs = static_cast<uint32_t>(__shfl_xor(static_cast<int>(high ? c[j] : c[4 + j]), 2));
    *gmem(blk + L::v_off(t, q, d16 + j)) = static_cast<uint8_t>(high ? theirs | mine << 4 : mine | theirs << 4);
  }
  if (l8 == 0) {
    *gmem(reinterpret_cast<_Float16*>(blk + L::p_off(t, gr, 2))) = s16;
    *gmem(reinterpret_cast<_Float16*>(blk + L::p_off(t, gr, 3))) = z16;
  }
}

template <int D, int DT>
__global__ __launch_bounds__(kKv4Threads) void kv4_read_kernel(Kv4Geom g, Kv4Rows r) {
  using L = Kv4Layout<D>;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kKv4Threads + threadIdx.x) >> 3;
  const int l8 = threadIdx.x & 7;
  const int gr = static_cast<int>(unit % L::kGroups);
  const int64_t th = unit / L::kGroups;
  const int64_t tok = th / g.n_kv_heads;
  if (tok >= r.n) return;
  const int head = static_cast<int>(th - tok * g.n_kv_heads);
  const int64_t slot = gmem(r.slots)[tok];
  const int64_t page = slot >> g.page_shift;
  float kx[8], vx[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) kx[j] = vx[j] = 0.0f;
  if (slot >= 0 && page < g.n_pages) {
    const int in_page = static_cast<int>(slot & ((1 << g.page_shift) - 1));
    const int t = in_page & (kKv4Block - 1);
    const uint8_t* blk = g.data + kv4_block_off<D>(g, page, head, in_page / kKv4Block);
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = static_cast<float>(*gmem(reinterpret_cast<const _Float16*>(blk + L::p_off(t, gr, i))));
    const u32x2_t w = *gmem(reinterpret_cast<const u32x2_t*>(blk + L::k_off(t, gr, l8 & 3)));
    const int ksh = l8 & 4;
    const int q = 2 * gr + (l8 >> 2), vsh = (l8 & 2) << 1, d16 = (l8 & 1) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t kc = (w[j >> 2] >> (8 * kv4_byte(j & 3) + ksh)) & 15u;
      const uint32_t vc = (static_cast<uint32_t>(*gmem(blk + L::v_off(t, q, d16 + j))) >> vsh) & 15u;
      kx[j] = __builtin_fmaf(p[0], static_cast<float>(kc), p[1]);
      vx[j] = __builtin_fmaf(p[2], static_cast<float>(vc), p[3]);
    }
  }
  store8<DT>(r.k_out, tok * r.k_st + head * r.k_sh + gr * kKv4Group + 8 * l8, kx);
  store8<DT>(r.v_out, tok * r.v_st + head * r.v_sh + gr * kKv4Group + 8 * l8, vx);
}

template <int D, int DT>
void launch_rows(const Kv4Geom& g, const Kv4Rows& r, bool write, hipStream_t stream) {
  const int64_t lanes = r.n * g.n_kv_heads * Kv4Layout<D>::kGroups * 8;
  const dim3 grid(static_cast<unsigned>((lanes + kKv4Threads - 1) / kKv4Threads));
  if (write)
    hipLaunchKernelGGL((kv4_write_kernel<D, DT>), grid, dim3(kKv4Threads), 0, stream, g, r);
  else
    hipLaunchKernelGGL((kv4_read_kernel<D, DT>), grid, dim3(kKv4Threads), 0, stream, g, r);
}

template <int D>
void launch_dt(const Kv4Geom& g, const Kv4Rows& r, int dt, bool write, hipStream_t stream) {
  if (dt == kActF32)
    launch_rows<D, kActF32>(g, r, write, stream);
  else if (dt == kActF16)
    launch_rows<D, kActF16>(g, r, write, stream);
  else
    launch_rows<D, kActBf16>(g, r, write, stream);
}

}  // namespace

hipError_t launch_kv4_rows(const Kv4Geom& g, int head_dim, const Kv4Rows& r, int dt, bool write, hipStream_t stream) {
  if (head_dim == 64)
    launch_dt<64>(g, r, dt, write, stream);
  else
    launch_dt<128>(g, r, dt, write, stream);
  return hipGetLastError();
}

}  // namespace sherry
