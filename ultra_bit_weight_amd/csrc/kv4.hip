// Writing keys and values into the 4-bit cache, and reading them back.
//
// For 64 consecutive values x of one token and head:
//   z = f16(min x), s = f16((max x - min x) / 15), clamped to +-65504
//   c = clip(rint((x - z) / s), 0, 15), 0 where s = 0     (IEEE fp32 steps)
//   value = z + s c                                       (one fp32 rounding)
//
// Eight lanes take a group, eight values each: the extremes are one three-step
// DPP reduction, and a lane's codes are whole nibbles of the layout's dwords.
//
// A workgroup takes 32 tokens of one head.  When their slots are one whole block
// (a prompt chunk: the tiles are cut where the first token's slot says blocks
// begin), the block passes through LDS and memory sees 16-byte accesses only;
// else each token's bytes are written or read where they lie.
// Bound: HBM (K and V are read once, a quarter of them written, or the reverse):
// 20011 tokens of 8 heads of 64 read back in 10.0 us, 5.3 TB/s, the rate of a
// large copy; 8192 tokens of 8 heads of 128 written in about 14 us, 3.0 TB/s,
// where the quantiser's arithmetic (20 instructions a value, of them 6 the exact
// quotient) is half the time: the vector unit is 43 % busy, and a wave waits for
// half of its life, since a workgroup's load, arithmetic and store follow one
// another and the eight of a CU begin together.
#include "kv4.h"

namespace sherry {
namespace {

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

// The group's values that a lane restores: 8 l8 .. + 7 of K and of V.
template <int D, class B>
__device__ __forceinline__ void get_kv(const B* blk, int t, int gr, int l8, float (&kx)[8], float (&vx)[8]) {
  using L = Kv4Layout<D>;
  float p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = static_cast<float>(*gmem_or_lds<const _Float16>(blk + L::p_off(t, gr, i)));
  const u32x2_t w = *gmem_or_lds<const u32x2_t>(blk + L::k_off(t, gr, l8 & 3));
  const int ksh = l8 & 4, q = 2 * gr + (l8 >> 2), vsh = (l8 & 2) << 1, d16 = (l8 & 1) * 8;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t kc = (w[j >> 2] >> (8 * kv4_byte(j & 3) + ksh)) & 15u;
    const uint32_t vc = (static_cast<uint32_t>(*gmem_or_lds<const uint8_t>(blk + L::v_off(t, q, d16 + j))) >> vsh) & 15u;
    kx[j] = __builtin_fmaf(p[0], static_cast<float>(kc), p[1]);
    vx[j] = __builtin_fmaf(p[2], static_cast<float>(vc), p[3]);
  }
}

// A thread's tasks: lane l8 of group gr of token place t, `kTasks` of them.
template <int D, int DT>
__global__ __launch_bounds__(kKv4Threads) void kv4_write_kernel(Kv4Geom g, Kv4Rows r) {
  using L = Kv4Layout<D>;
  constexpr int kTasks = kKv4Block * L::kGroups * 8 / kKv4Threads;
  __shared__ u32x4_t image[L::kBytes / 16];
  const int number = blockIdx.x / g.n_kv_heads, head = blockIdx.x - number * g.n_kv_heads;
  const int64_t first = tile_first(r, number);
  const int64_t slot = tile_slot(r, first);  // K and V are under way before it is looked at
  const int l8 = threadIdx.x & 7;
  float kx[kTasks][8], vx[kTasks][8];
#pragma unroll
  for (int i = 0; i < kTasks; ++i) {
    const int u = (threadIdx.x + i * kKv4Threads) >> 3, gr = u % L::kGroups;
    const int64_t tok = first + u / L::kGroups;
    if (tok >= 0 && tok < r.n) {
      load8<DT>(r.k, tok * r.k_st + head * r.k_sh + gr * kKv4Group + 8 * l8, kx[i]);
      load8<DT>(r.v, tok * r.v_st + head * r.v_sh + gr * kKv4Group + 8 * l8, vx[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) kx[i][j] = vx[i][j] = 0.0f;
    }
  }
  uint8_t* block = tile_block<D>(g, slot, head);
#pragma unroll
  for (int i = 0; i < kTasks; ++i) {
    const int u = (threadIdx.x + i * kKv4Threads) >> 3, gr = u % L::kGroups, place = u / L::kGroups;
    const int64_t tok = first + place;
    u32x2_t kc, vc;
    _Float16 ks, kz, vs, vz;
    quantise8(kx[i], &kc, &ks, &kz);
    quantise8(vx[i], &vc, &vs, &vz);
    if (block) {
      auto* blk = reinterpret_cast<SHERRY_LDS uint8_t*>((SHERRY_LDS u32x4_t*)image);
      put_k<D>(blk, place, gr, l8, kc, ks, kz);
      put_v<D>(blk, place, gr, l8, vc, vs, vz);
    } else if (tok >= 0 && tok < r.n) {  // (all eight lanes or none)
      int t;
      uint8_t* at = slot_block<D>(g, gmem(r.slots)[tok], head, &t);
      if (at) {
        put_k<D>(gmem(at), t, gr, l8, kc, ks, kz);
        put_v<D>(gmem(at), t, gr, l8, vc, vs, vz);
      }
    }
  }
  if (!block) return;
  __syncthreads();
  for (int i = threadIdx.x; i < L::kBytes / 16; i += kKv4Threads)
    *gmem(reinterpret_cast<u32x4_t*>(block) + i) = image[i];
}

template <int D, int DT, bool kStream>
__global__ __launch_bounds__(kKv4Threads) void kv4_read_kernel(Kv4Geom g, Kv4Rows r) {
  using L = Kv4Layout<D>;
  constexpr int kTasks = kKv4Block * L::kGroups * 8 / kKv4Threads;
  __shared__ u32x4_t image[L::kBytes / 16];
  const int number = blockIdx.x / g.n_kv_heads, head = blockIdx.x - number * g.n_kv_heads;
  const int64_t first = tile_first(r, number);
  uint8_t* block = tile_block<D>(g, tile_slot(r, first), head);
  const int l8 = threadIdx.x & 7;
  if (block) {
    for (int i = threadIdx.x; i < L::kBytes / 16; i += kKv4Threads)
      image[i] = *gmem(reinterpret_cast<const u32x4_t*>(block) + i);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kTasks; ++i) {
    const int u = (threadIdx.x + i * kKv4Threads) >> 3, gr = u % L::kGroups, place = u / L::kGroups;
    const int64_t tok = first + place;
    if (tok < 0 || tok >= r.n) continue;
    float kx[8], vx[8];
    if (block) {
      get_kv<D>(reinterpret_cast<const SHERRY_LDS uint8_t*>((const SHERRY_LDS u32x4_t*)image), place, gr, l8, kx, vx);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) kx[j] = vx[j] = 0.0f;
      int t;
      const uint8_t* at = slot_block<D>(g, gmem(r.slots)[tok], head, &t);
      if (at) get_kv<D>(gmem(at), t, gr, l8, kx, vx);
    }
    store8<DT, kStream>(r.k_out, tok * r.k_st + head * r.k_sh + gr * kKv4Group + 8 * l8, kx);
    store8<DT, kStream>(r.v_out, tok * r.v_st + head * r.v_sh + gr * kKv4Group + 8 * l8, vx);
  }
}

template <int D, int DT>
void launch_rows(const Kv4Geom& g, const Kv4Rows& r, bool write, hipStream_t stream) {
  // one tile more than n / 32: the first may begin up to 31 tokens before token
  // 0; a tile's heads are neighbours, and so is what they read
  const dim3 grid(static_cast<unsigned>((r.n + 2 * kKv4Block - 2) / kKv4Block * g.n_kv_heads));
  if (write)
    hipLaunchKernelGGL((kv4_write_kernel<D, DT>), grid, dim3(kKv4Threads), 0, stream, g, r);
  else if (2 * r.n * g.n_kv_heads * D * act_bytes(DT) > kStreamBytes)
    hipLaunchKernelGGL((kv4_read_kernel<D, DT, true>), grid, dim3(kKv4Threads), 0, stream, g, r);
  else
    hipLaunchKernelGGL((kv4_read_kernel<D, DT, false>), grid, dim3(kKv4Threads), 0, stream, g, r);
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
