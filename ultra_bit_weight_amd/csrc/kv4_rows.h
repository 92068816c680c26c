// Rows of the 4-bit cache in and out: the quantiser and the places of a token's
// codes and scales, shared by the cache's write and read (kv4.hip) and the append
// with norms and rotation (kv4_append.hip).  Eight lanes take a group of 64
// values, eight values each.
#pragma once

#include "kv4.h"

namespace sherry {

constexpr int kKv4Threads = 256;

#define SHERRY_LDS __attribute__((address_space(3)))
// A typed access at a byte of device memory or of LDS, in its address space.
template <class T>
__device__ __forceinline__ SHERRY_GLOBAL T* gmem_or_lds(SHERRY_GLOBAL uint8_t* p) {
  return reinterpret_cast<SHERRY_GLOBAL T*>(p);
}
template <class T>
__device__ __forceinline__ const SHERRY_GLOBAL T* gmem_or_lds(const SHERRY_GLOBAL uint8_t* p) {
  return reinterpret_cast<const SHERRY_GLOBAL T*>(p);
}
template <class T>
__device__ __forceinline__ SHERRY_LDS T* gmem_or_lds(SHERRY_LDS uint8_t* p) {
  return reinterpret_cast<SHERRY_LDS T*>(p);
}
template <class T>
__device__ __forceinline__ const SHERRY_LDS T* gmem_or_lds(const SHERRY_LDS uint8_t* p) {
  return reinterpret_cast<const SHERRY_LDS T*>(p);
}

__device__ __forceinline__ float f16_clamped(float v, _Float16* h) {
  *h = static_cast<_Float16>(fminf(fmaxf(v, -65504.0f), 65504.0f));
  return static_cast<float>(*h);
}

template <int CTRL>
__device__ __forceinline__ float dpp_of(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, false));
}

// min and max of three as the instructions (fminf first quiets every operand).
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// a / b, correctly rounded, from inv = 1 / b correctly rounded: t = a inv is
// within an ulp, a - t b is exact, and t + (a - t b) inv rounds to the quotient
// (Markstein's theorem; every b here has few bits, so never 24 ones, and both
// are far from the ends of the range).
__device__ __forceinline__ float quotient(float a, float b, float inv) {
  const float t = a * inv;
  return __builtin_fmaf(__builtin_fmaf(-t, b, a), inv, t);
}

// Codes of the lane's eight values, four to a dword in the layout's byte order;
// the eight lanes of a group share s and z.
__device__ __forceinline__ void quantise8(const float (&v)[8], u32x2_t* codes, _Float16* s16, _Float16* z16) {
  float lo = min3(min3(min3(v[0], v[1], v[2]), v[3], v[4]), min3(v[5], v[6], v[7]), v[0]);
  float hi = max3(max3(max3(v[0], v[1], v[2]), v[3], v[4]), max3(v[5], v[6], v[7]), v[0]);
  const float lo1 = dpp_of<0xB1>(lo), hi1 = dpp_of<0xB1>(hi);  // quad_perm [1,0,3,2]
  lo = min3(lo, lo1, lo1), hi = max3(hi, hi1, hi1);
  const float lo2 = dpp_of<0x4E>(lo), hi2 = dpp_of<0x4E>(hi);  // quad_perm [2,3,0,1]
  lo = min3(lo, lo2, lo2), hi = max3(hi, hi2, hi2);
  const float lo3 = dpp_of<0x141>(lo), hi3 = dpp_of<0x141>(hi);  // row_half_mirror
  lo = min3(lo, lo3, lo3), hi = max3(hi, hi3, hi3);
  const float z = f16_clamped(lo, z16);
  // (a range past 15 * 65504 ends at the same s)
  const float s = f16_clamped(quotient(fminf(hi - lo, 1.0e6f), 15.0f, 1.0f / 15.0f), s16);
  // 1 / s: one Newton step from the hardware's reciprocal, correctly rounded for
  // every positive fp16 s
  const float r0 = __builtin_amdgcn_rcpf(s);
  const float inv = s > 0.0f ? __builtin_fmaf(__builtin_fmaf(-s, r0, 1.0f), r0, r0) : 0.0f;
  // Clipping before rounding is the same as after, and adding 1.5 * 2^23 rounds
  // half to even and leaves the integer in the low byte.
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    c[j] = __float_as_uint(__builtin_amdgcn_fmed3f(quotient(v[j] - z, s, inv), 0.0f, 15.0f) + 12582912.0f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // bytes 0, 1, 2, 3 from values 0, 2, 1, 3
    const uint32_t even = __builtin_amdgcn_perm(c[4 * i + 1], c[4 * i], 0x0C040C00u);
    const uint32_t odd = __builtin_amdgcn_perm(c[4 * i + 3], c[4 * i + 2], 0x040C000Cu);
    (*codes)[i] = even | odd;
  }
}

// First token of a tile (those before 0 or past the last do not exist).
__device__ __forceinline__ int64_t tile_first(const Kv4Rows& r, int number) {
  return static_cast<int64_t>(number) * kKv4Block - (gmem(r.slots)[0] & (kKv4Block - 1));
}
// A slot of the tile, each wave's lanes all 32 of them (-1 past the ends).
__device__ __forceinline__ int64_t tile_slot(const Kv4Rows& r, int64_t first) {
  const int64_t i = first + (threadIdx.x & (kKv4Block - 1));
  return i >= 0 && i < r.n ? gmem(r.slots)[i] : -1;
}
// The block that the tile's slots are, or null.
template <int D>
__device__ __forceinline__ uint8_t* tile_block(const Kv4Geom& g, int64_t slot, int head) {
  const int64_t s0 = __shfl(slot, 0);
  const bool run = slot == s0 + (threadIdx.x & (kKv4Block - 1)) && (s0 & (kKv4Block - 1)) == 0 && s0 >= 0 &&
                   (s0 >> g.page_shift) < g.n_pages;
  if (!__all(run)) return nullptr;
  const int in_page = static_cast<int>(s0 & ((1 << g.page_shift) - 1));
  return g.data + kv4_block_off<D>(g, s0 >> g.page_shift, head, in_page / kKv4Block);
}

// Block and place of one token's slot; null for none.
template <int D>
__device__ __forceinline__ uint8_t* slot_block(const Kv4Geom& g, int64_t slot, int head, int* t) {
  const int64_t page = slot >> g.page_shift;
  if (slot < 0 || page >= g.n_pages) return nullptr;
  const int in_page = static_cast<int>(slot & ((1 << g.page_shift) - 1));
  *t = in_page & (kKv4Block - 1);
  return g.data + kv4_block_off<D>(g, page, head, in_page / kKv4Block);
}

// K codes and scales of one group to a block in LDS or in memory: low nibbles
// come from lanes 0-3 of the eight, high ones from 4-7.
template <int D, class B>
__device__ __forceinline__ void put_k(B* blk, int t, int gr, int l8, u32x2_t w, _Float16 s, _Float16 z) {
  using L = Kv4Layout<D>;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] |= static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(w[i]), 0x104, 0xF, 0xF, false)) << 4;  // row_shl:4
  if (l8 < 4) *gmem_or_lds<u32x2_t>(blk + L::k_off(t, gr, l8)) = w;
  if (l8 == 0) *gmem_or_lds<_Float16>(blk + L::p_off(t, gr, 0)) = s;
  if (l8 == 1) *gmem_or_lds<_Float16>(blk + L::p_off(t, gr, 1)) = z;
}

// V: a byte holds two values 16 apart, so lanes two apart share bytes; each of
// the two stores four of their eight.
template <int D, class B>
__device__ __forceinline__ void put_v(B* blk, int t, int gr, int l8, u32x2_t c, _Float16 s, _Float16 z) {
  using L = Kv4Layout<D>;
  const bool high = l8 & 2;
  const int q = 2 * gr + (l8 >> 2), d16 = (l8 & 1) * 8 + (high ? 4 : 0);
  const int give = static_cast<int>(high ? c.x : c.y);
  const uint32_t theirs = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(give, give, 0x4E, 0xF, 0xF, false));
  const uint32_t w = high ? theirs | c.y << 4 : c.x | theirs << 4;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *gmem_or_lds<uint8_t>(blk + L::v_off(t, q, d16 + j)) = static_cast<uint8_t>(w >> (8 * kv4_byte(j)));
  if (l8 == 2) *gmem_or_lds<_Float16>(blk + L::p_off(t, gr, 2)) = s;
  if (l8 == 3) *gmem_or_lds<_Float16>(blk + L::p_off(t, gr, 3)) = z;
}

}  // namespace sherry
