// New tokens into the 4-bit cache: norms and rotation of q and k, k and v
// quantised where they are used last, in one launch (what qk_norm_rope followed
// by the cache's write does in two, without the 16-bit k between them).
//
//   n = x rsqrt(mean(x^2) + eps) w, rotation of its first rot values   (rope.h)
//   k and v per 64 values: z = f16(min), s = f16((max - min) / 15),
//     c = clip(rint((x - z) / s), 0, 15)                               (kv4_rows.h)
//
// The first workgroups take 32 tokens of one key head each: k is normalised and
// rotated in the lanes that hold whole pairs, and passes through LDS as fp32 to
// the lanes that quantise, so that not a bit differs from the two steps with an
// fp32 k between them.  The others take q as the rotation alone does.
#include "kv4_rows.h"
#include "rope.h"

namespace sherry {
namespace {

template <int D, int XDT, int YDT>
__global__ __launch_bounds__(kKv4Threads) void kv4_append_kernel(Kv4Geom g, RopeArgs a, Kv4Rows r, int kv_blocks) {
  using L = Kv4Layout<D>;
  constexpr int kTasks = kKv4Block * L::kGroups * 8 / kKv4Threads;
  constexpr int kLph = D / 16;  // lanes of a head in the rotation
  constexpr int kPad = D + 4;
  __shared__ u32x4_t image[L::kBytes / 16];
  __shared__ float lds_k[kKv4Block * kPad];
  if (static_cast<int>(blockIdx.x) >= kv_blocks) {  // q
    const uint32_t unit = ((blockIdx.x - kv_blocks) * static_cast<uint32_t>(kKv4Threads) + threadIdx.x) / kLph;
    const uint32_t tok = unit / a.q.heads, head = unit - tok * a.q.heads;
    const bool has = tok < a.n;
    float x0[1][8], x1[1][8];
    int d0, d1;
    norm_rope<XDT, 1>(a, a.q, tok, head, threadIdx.x & (kLph - 1), has, x0, x1, d0, d1);
    if (!has) return;
    const int64_t to = tok * a.q.y_st + head * a.q.y_sh;
    store8<YDT>(a.q.y, to + d0, x0[0]);
    store8<YDT>(a.q.y, to + d1, x1[0]);
    return;
  }
  const int number = blockIdx.x / g.n_kv_heads, head = blockIdx.x - number * g.n_kv_heads;
  const int64_t first = tile_first(r, number);
  // a token whose position has no angles is not written
  int64_t slot = tile_slot(r, first);
  if (slot >= 0) {
    const int64_t pos = gmem(a.pos)[first + (threadIdx.x & (kKv4Block - 1))];
    if (pos < 0 || pos >= a.max_pos) slot = -1;
  }
  const int l8 = threadIdx.x & 7;
  float vx[kTasks][8];
#pragma unroll
  for (int i = 0; i < kTasks; ++i) {
    const int u = (threadIdx.x + i * kKv4Threads) >> 3, gr = u % L::kGroups;
    const int64_t tok = first + u / L::kGroups;
#pragma unroll
    for (int j = 0; j < 8; ++j) vx[i][j] = 0.0f;
    if (tok >= 0 && tok < r.n) load8<XDT>(r.v, tok * r.v_st + head * r.v_sh + gr * kKv4Group + 8 * l8, vx[i]);
  }
  if (threadIdx.x < kKv4Block * kLph) {
    const int place = threadIdx.x / kLph;
    const int64_t tok = first + place;
    const bool has = tok >= 0 && tok < a.n;
    float x0[1][8], x1[1][8];
    int d0, d1;
    norm_rope<XDT, 1>(a, a.k, tok, head, threadIdx.x & (kLph - 1), has, x0, x1, d0, d1);
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      *reinterpret_cast<f32x4_t*>(&lds_k[place * kPad + d0 + j]) = f32x4_t{x0[0][j], x0[0][j + 1], x0[0][j + 2], x0[0][j + 3]};
      *reinterpret_cast<f32x4_t*>(&lds_k[place * kPad + d1 + j]) = f32x4_t{x1[0][j], x1[0][j + 1], x1[0][j + 2], x1[0][j + 3]};
    }
  }
  uint8_t* block = tile_block<D>(g, slot, head);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTasks; ++i) {
    const int u = (threadIdx.x + i * kKv4Threads) >> 3, gr = u % L::kGroups, place = u / L::kGroups;
    float kx[8];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const f32x4_t t = *reinterpret_cast<const f32x4_t*>(&lds_k[place * kPad + gr * kKv4Group + 8 * l8 + j]);
      kx[j] = t.x, kx[j + 1] = t.y, kx[j + 2] = t.z, kx[j + 3] = t.w;
    }
    u32x2_t kc, vc;
    _Float16 ks, kz, vs, vz;
    quantise8(kx, &kc, &ks, &kz);
    quantise8(vx[i], &vc, &vs, &vz);
    const int64_t own_slot = __shfl(slot, place);
    if (block) {
      auto* blk = reinterpret_cast<SHERRY_LDS uint8_t*>((SHERRY_LDS u32x4_t*)image);
      put_k<D>(blk, place, gr, l8, kc, ks, kz);
      put_v<D>(blk, place, gr, l8, vc, vs, vz);
    } else {
      int t;
      uint8_t* at = slot_block<D>(g, own_slot, head, &t);
      if (at) {  // (all eight lanes or none)
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

template <int D, int XDT, int YDT>
void launch_xy(const Kv4Geom& g, const RopeArgs& a, const Kv4Rows& r, hipStream_t stream) {
  const int64_t kv = (r.n + 2 * kKv4Block - 2) / kKv4Block * g.n_kv_heads;
  const int64_t q = (a.n * a.q.heads * (D / 16) + kKv4Threads - 1) / kKv4Threads;
  hipLaunchKernelGGL((kv4_append_kernel<D, XDT, YDT>), dim3(static_cast<unsigned>(kv + q)), dim3(kKv4Threads), 0, stream,
                     g, a, r, static_cast<int>(kv));
}

template <int D, int XDT>
void launch_x(const Kv4Geom& g, const RopeArgs& a, const Kv4Rows& r, int ydt, hipStream_t stream) {
  if (ydt == kActF32)
    launch_xy<D, XDT, kActF32>(g, a, r, stream);
  else if (ydt == kActF16)
    launch_xy<D, XDT, kActF16>(g, a, r, stream);
  else
    launch_xy<D, XDT, kActBf16>(g, a, r, stream);
}

template <int D>
void launch_d(const Kv4Geom& g, const RopeArgs& a, const Kv4Rows& r, int xdt, int ydt, hipStream_t stream) {
  if (xdt == kActF32)
    launch_x<D, kActF32>(g, a, r, ydt, stream);
  else if (xdt == kActF16)
    launch_x<D, kActF16>(g, a, r, ydt, stream);
  else
    launch_x<D, kActBf16>(g, a, r, ydt, stream);
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Geom& g, int head_dim, const RopeArgs& a, const Kv4Rows& r, int xdt, int ydt,
                             hipStream_t stream) {
  if (head_dim == 64)
    launch_d<64>(g, a, r, xdt, ydt, stream);
  else
    launch_d<128>(g, a, r, xdt, ydt, stream);
  return hipGetLastError();
}

}  // namespace sherry
