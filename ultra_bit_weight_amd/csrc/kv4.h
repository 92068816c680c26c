// Layout and device helpers of the 4-bit key/value cache (documented in
// include/sherry.h), shared by its write, read and attention kernels.
//
// The unit is a block: 32 consecutive tokens of one page and one head, K and V
// codes and their scales together, so an attention wave streams whole blocks
// with 16-byte loads whose bytes are matrix-core operands as they lie: no
// shuffle and no LDS between HBM and the product.
#pragma once

#include "launch.h"

namespace sherry {

constexpr int kKv4Block = 32;  // tokens per block
constexpr int kKv4Group = 64;  // values per scale

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Byte of a dword that holds value i (0..3): the masked halves of the dword
// and of the dword >> 8 are then the pairs (0, 1) and (2, 3).
__host__ __device__ constexpr int kv4_byte(int i) { return ((i & 1) << 1) | (i >> 1); }

template <int D>
struct Kv4Layout {
  static constexpr int kGroups = D / kKv4Group;
  static constexpr int kVOff = 16 * D;         // V codes
  static constexpr int kPOff = 32 * D;         // scales and zero points
  static constexpr int kBytes = 32 * D + 256 * kGroups;

  // 8 K bytes (16 codes: values 64 gr + 8 g .. + 7 in the low nibbles,
  // 64 gr + 32 + 8 g .. + 7 in the high ones) of token t of the block
  __host__ __device__ static constexpr int k_off(int t, int gr, int g) {
    const int tile = t >> 4, t16 = t & 15;
    return D == 64 ? ((g * 16 + t16) * 2 + tile) * 8 : ((tile * 4 + g) * 16 + t16) * 16 + gr * 8;
  }
  // the V byte of token t that holds values 32 q + d16 (low) and
  // 32 q + 16 + d16 (high)
  __host__ __device__ static constexpr int v_off(int t, int q, int d16) {
    const int tile = t >> 4, g = (t >> 2) & 3;
    return kVOff + (q >> 1) * 1024 + (g * 16 + d16) * 16 + (q & 1) * 8 + tile * 4 + kv4_byte(t & 3);
  }
  // fp16 parameter `which` (0 K scale, 1 K zero, 2 V scale, 3 V zero) of token
  // t, group gr
  __host__ __device__ static constexpr int p_off(int t, int gr, int which) {
    const int tile = t >> 4, g = (t >> 2) & 3;
    return kPOff + gr * 256 + which * 64 + g * 16 + tile * 8 + (t & 3) * 2;
  }
};

template <int D>
__device__ __forceinline__ int64_t kv4_block_off(const Kv4Geom& c, int64_t page, int head, int block) {
  return (((page * c.n_kv_heads + head) << (c.page_shift - 5)) + block) * Kv4Layout<D>::kBytes;
}

// Eight consecutive values as fp32 (16-byte loads; the host checks alignment).
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (DT == kActF32) {
    const f32x4_t a = *gmem(reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i));
    const f32x4_t b = *gmem(reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i + 4));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
  } else {
    const u32x4_t w = *gmem(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + i));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = (w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
      v[j] = DT == kActF16 ? static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)))
                           : __uint_as_float(h << 16);
    }
  }
}

// Two fp32 rounded to nearest even as a pair of 16-bit values.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == kActF16) {
    const half2_t h = {static_cast<_Float16>(a), static_cast<_Float16>(b)};
    return __builtin_bit_cast(uint32_t, h);
  } else {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    const bf2 h = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, h);
  }
}

// kStream: past the caches (for outputs larger than they are).
template <int DT, bool kStream = false>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  auto put = [](auto w, auto* to) {
    if constexpr (kStream)
      __builtin_nontemporal_store(w, to);
    else
      *to = w;
  };
  if constexpr (DT == kActF32) {
    f32x4_t a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = v[j], b[j] = v[4 + j];
    put(a, gmem(reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i)));
    put(b, gmem(reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i + 4)));
  } else {
    u32x4_t w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack2<DT>(v[2 * j], v[2 * j + 1]);
    put(w, gmem(reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i)));
  }
}

// Outputs of more bytes than this are stored past the caches: the L2s hold 32
// MB, shared with the inputs.  Measured: norms and rotation of 67 MB 38.1 ->
// 25.5 us, reading 20011 tokens back (41 MB) 10.8 -> 10.0 us.
constexpr int64_t kStreamBytes = int64_t(16) << 20;
inline int64_t act_bytes(int dt) { return dt == kActF32 ? 4 : 2; }

}  // namespace sherry
