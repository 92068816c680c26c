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
#include "kv4_rows.h"

namespace sherry {
namespace {

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
