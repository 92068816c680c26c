// New tokens into the 4-bit cache: norms and rotation of q and k, k and v
// quantised, in one launch (what qk_norm_rope followed by the cache's write does in
// two, without the 16-bit k between them).
//
//   n = x rsqrt(mean(x^2) + eps) w, rotation of its first rot values   (rope.h)
//   k and v per 64 values: z = f16(min), s = f16((max - min) / 15),
//     c = clip(rint((x - z) / s), 0, 15)                               (kv4_rows.h)
//
// Some workgroups take 32 tokens of one key head each, the others q as the rotation
// alone does, in turn over the launch, so that the quantiser's arithmetic runs under
// q's loads and stores.  Where all of a head rotates in half-split pairs, the lanes
// of the rotation hold what the quantiser wants together, and k never leaves their
// registers; otherwise it passes through LDS as fp32.  Either way not a bit differs
// from the two steps with an fp32 k between them.
//
// Bound by HBM, beside the quantiser's arithmetic: 8192 tokens of 24 + 8 heads of 128
// in 16 bits with norms 31-32 us, 4.6-4.7 TB/s (a large copy 5.1), the vector unit 58 %
// busy; the two steps apart 24.3 and 14.  One token 2.9 us: a launch, and the angles'
// load behind the position's.  No load stands behind a branch, which the compiler
// would wait for before the next (8192 tokens 36.5 us with them).
#include <type_traits>

#include "kv4_rows.h"
#include "rope.h"

namespace sherry {
namespace {

struct AppendArgs {
  Kv4Geom g;
  RopeArgs a;
  Kv4Rows r;
  uint32_t kv_blocks;  // workgroups of k and v,
  uint32_t kv_share;   // (i * kv_share) >> 32 of them before workgroup i; 0: they go first
  int32_t stream;      // q past the caches
};

// q: HPL heads a lane
template <int D, int XDT, int YDT, int HPL, bool kDirect>
__device__ __forceinline__ void append_q(const AppendArgs& p, uint32_t number) {
  constexpr int kLph = D / 16;
  const RopeArgs& a = p.a;
  const uint32_t unit = (number * static_cast<uint32_t>(kKv4Threads) + threadIdx.x) / kLph;
  const uint32_t sets = (a.q.heads + HPL - 1) / HPL;
  const uint32_t tok = unit / sets;
  const int head = static_cast<int>((unit - tok * sets) * HPL);
  const bool has = tok < a.n;
  float x0[HPL][8], x1[HPL][8];
  int d0, d1;
  norm_rope<XDT, HPL, true, kDirect>(a, a.q, min(static_cast<int64_t>(tok), a.n - 1), head, threadIdx.x & (kLph - 1), true,
                                     x0, x1, d0, d1);
  if (!has) return;
  auto store = [&](auto past) {
#pragma unroll
    for (int h = 0; h < HPL; ++h) {
      if (head + h >= a.q.heads) break;
      const int64_t to = tok * a.q.y_st + (head + h) * a.q.y_sh;
      store8<YDT, decltype(past)::value>(a.q.y, to + d0, x0[h]);
      store8<YDT, decltype(past)::value>(a.q.y, to + d1, x1[h]);
    }
  };
  if (p.stream)
    store(std::true_type{});
  else
    store(std::false_type{});
}

template <int D, int XDT, int YDT, int HPL, bool kDirect>
__global__ __launch_bounds__(kKv4Threads) void kv4_append_kernel(AppendArgs p) {
  using L = Kv4Layout<D>;
  constexpr int kLph = D / 16;                                              // lanes of a head in the rotation
  constexpr int kPlaces = kKv4Threads / 8;                                  // tokens of eight lanes each
  static_assert(kPlaces == kKv4Block && kKv4Block * kLph <= kKv4Threads);
  constexpr int kPad = D + 4;
  __shared__ u32x4_t image[L::kBytes / 16];
  __shared__ float lds_k[kDirect ? 1 : kKv4Block * kPad];
  auto upto = [&](uint32_t i) { return min(p.kv_share ? __umulhi(i, p.kv_share) : i, p.kv_blocks); };
  const uint32_t before = upto(blockIdx.x);
  if (upto(blockIdx.x + 1) == before) return append_q<D, XDT, YDT, HPL, kDirect>(p, blockIdx.x - before);
  const Kv4Geom& g = p.g;
  const RopeArgs& a = p.a;
  const Kv4Rows& r = p.r;
  const int number = before / g.n_kv_heads, head = before - number * g.n_kv_heads;
  const int64_t first = tile_first(r, number);
  const int l8 = threadIdx.x & 7, place = threadIdx.x >> 3;
  // Places of no token load the nearest one's values (no load behind a branch) and
  // have no slot, as tokens whose position has no angles.
  auto token = [&](int at) { return min(max(first + at, int64_t(0)), r.n - 1); };
  const int at_lane = threadIdx.x & (kKv4Block - 1);
  int64_t slot = gmem(r.slots)[token(at_lane)];
  const int64_t pos = gmem(a.pos)[token(at_lane)];
  const int64_t tok = token(place);
  float vx[L::kGroups][8];
#pragma unroll
  for (int i = 0; i < L::kGroups; ++i)
    load8<XDT>(r.v, tok * r.v_st + head * r.v_sh + i * kKv4Group + 8 * l8, vx[i]);
  float kx[L::kGroups][8];
  {
    float x0[1][8], x1[1][8];
    int d0, d1;
    if constexpr (kDirect && D == 128) {  // the two runs are run l8 of either group
      norm_rope<XDT, 1, true, true>(a, a.k, tok, head, l8, true, x0, x1, d0, d1);
#pragma unroll
      for (int j = 0; j < 8; ++j) kx[0][j] = x0[0][j], kx[L::kGroups - 1][j] = x1[0][j];
    } else if constexpr (kDirect) {  // the two runs are runs l8 % 4 and l8 % 4 + 4: each lane of a pair keeps one
      norm_rope<XDT, 1, true, true>(a, a.k, tok, head, l8 & 3, true, x0, x1, d0, d1);
#pragma unroll
      for (int j = 0; j < 8; ++j) kx[0][j] = l8 < 4 ? x0[0][j] : x1[0][j];
    } else {
      if (threadIdx.x < kKv4Block * kLph) {
        const int at = threadIdx.x / kLph;
        norm_rope<XDT, 1, true>(a, a.k, token(at), head, threadIdx.x & (kLph - 1), true, x0, x1, d0, d1);
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          *reinterpret_cast<f32x4_t*>(&lds_k[at * kPad + d0 + j]) = f32x4_t{x0[0][j], x0[0][j + 1], x0[0][j + 2], x0[0][j + 3]};
          *reinterpret_cast<f32x4_t*>(&lds_k[at * kPad + d1 + j]) = f32x4_t{x1[0][j], x1[0][j + 1], x1[0][j + 2], x1[0][j + 3]};
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < L::kGroups; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const f32x4_t t = *reinterpret_cast<const f32x4_t*>(&lds_k[place * kPad + i * kKv4Group + 8 * l8 + j]);
          kx[i][j] = t.x, kx[i][j + 1] = t.y, kx[i][j + 2] = t.z, kx[i][j + 3] = t.w;
        }
    }
  }
  if (first + at_lane < 0 || first + at_lane >= r.n || pos < 0 || pos >= a.max_pos) slot = -1;
  uint8_t* block = tile_block<D>(g, slot, head);
  const int64_t own_slot = __shfl(slot, place);
#pragma unroll
  for (int i = 0; i < L::kGroups; ++i) {
    u32x2_t kc, vc;
    _Float16 ks, kz, vs, vz;
    quantise8(kx[i], &kc, &ks, &kz);
    quantise8(vx[i], &vc, &vs, &vz);
    if (block) {
      auto* blk = reinterpret_cast<SHERRY_LDS uint8_t*>((SHERRY_LDS u32x4_t*)image);
      put_k<D>(blk, place, i, l8, kc, ks, kz);
      put_v<D>(blk, place, i, l8, vc, vs, vz);
    } else {
      int t;
      uint8_t* at = slot_block<D>(g, own_slot, head, &t);
      if (at) {  // (all eight lanes or none)
        put_k<D>(gmem(at), t, i, l8, kc, ks, kz);
        put_v<D>(gmem(at), t, i, l8, vc, vs, vz);
      }
    }
  }
  if (!block) return;
  __syncthreads();
  for (int i = threadIdx.x; i < L::kBytes / 16; i += kKv4Threads)
    *gmem(reinterpret_cast<u32x4_t*>(block) + i) = image[i];
}

// ---- few tokens: what counts is how long one wave's way is ----
//
// K and V, and the groups of 64 of a head, go to waves of their own, eight tokens
// each, so that no wave quantises twice; each token's bytes are written where they lie.
template <int D, int XDT, int YDT, bool kDirect>
__global__ __launch_bounds__(kKv4Threads) void kv4_append_few_kernel(AppendArgs p) {
  constexpr int kLph = D / 16, kPad = D + 4;
  constexpr int kWaves = kKv4Threads / kWave, kTokens = kWave / 8;
  constexpr int kSets = kWaves / (2 * Kv4Layout<D>::kGroups);  // of kTokens tokens
  __shared__ float lds_k[kDirect ? 1 : kWaves][kDirect ? 1 : kTokens * kPad];
  if (blockIdx.x >= p.kv_blocks) return append_q<D, XDT, YDT, 1, kDirect>(p, blockIdx.x - p.kv_blocks);
  const Kv4Geom& g = p.g;
  const RopeArgs& a = p.a;
  const Kv4Rows& r = p.r;
  const int number = blockIdx.x / g.n_kv_heads, head = blockIdx.x - number * g.n_kv_heads;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & (kWave - 1), place = lane >> 3, l8 = lane & 7;
  const bool is_v = wave & 1;
  const int gr = D == 64 ? 0 : wave >> 1;
  const int64_t first = (static_cast<int64_t>(number) * kSets + (D == 64 ? wave >> 1 : 0)) * kTokens;
  // (places of no token: the last one's values, and no slot)
  auto token = [&](int at) { return min(first + at, r.n - 1); };
  const int64_t tok = token(place);
  int64_t slot = gmem(r.slots)[tok];
  const int64_t pos = gmem(a.pos)[tok];
  float x[8];
  if (is_v) {
    load8<XDT>(r.v, tok * r.v_st + head * r.v_sh + gr * kKv4Group + 8 * l8, x);
  } else if (kDirect || lane < kTokens * kLph) {
    float x0[1][8], x1[1][8];
    int d0, d1;
    const int at = kDirect ? place : lane / kLph;
    norm_rope<XDT, 1, true, kDirect>(a, a.k, token(at), head, lane & (kLph - 1), true, x0, x1, d0, d1);
    if constexpr (kDirect) {
      // D = 128: the two runs are run l8 of either group; D = 64: runs l8 % 4 and l8 % 4 + 4
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = (D == 128 ? gr == 0 : l8 < 4) ? x0[0][j] : x1[0][j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) lds_k[wave][at * kPad + d0 + j] = x0[0][j], lds_k[wave][at * kPad + d1 + j] = x1[0][j];
    }
  }
  if constexpr (!kDirect) {
    __syncthreads();
    if (!is_v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = lds_k[wave][place * kPad + gr * kKv4Group + 8 * l8 + j];
    }
  }
  if (first + place >= r.n || pos < 0 || pos >= a.max_pos) slot = -1;
  u32x2_t c;
  _Float16 s, z;
  quantise8(x, &c, &s, &z);
  int t;
  uint8_t* to = slot_block<D>(g, slot, head, &t);
  if (!to) return;  // (all eight lanes of a token or none)
  if (is_v)
    put_v<D>(gmem(to), t, gr, l8, c, s, z);
  else
    put_k<D>(gmem(to), t, gr, l8, c, s, z);
}

// Heads of q a lane, where that leaves 1024 workgroups: 8192 tokens of 24 heads of 128
// 34.9 us with 1, 31.2 with 2, 31.4 with 4; of 32 heads of 64 20.1, 18.1, 18.5.
constexpr int kAppendHeads = 2;
constexpr int64_t kAtOnce = 2560;
// Up to this the few-token kernel: 1 token of 24 + 8 heads of 128 with norms 3.27 us,
// with the other kernel 4.36; 48 tokens 3.28, 4.57; 512 4.55, 5.28; 1000 7.27, 7.45; of
// 32 + 8 heads of 64 2.88, 3.25 (1), 3.31, 3.67 (512), 4.29, 4.50 (1000).
constexpr int64_t kFew = 1024;

template <int D, int XDT, int YDT>
void launch_xy(AppendArgs& p, hipStream_t stream) {
  const int64_t n = p.a.n;
  const dim3 block(kKv4Threads);
  const bool direct = p.a.rot == D && !p.a.interleaved;
  auto q_blocks = [&](int hpl) { return (n * ((p.a.q.heads + hpl - 1) / hpl) * (D / 16) + kKv4Threads - 1) / kKv4Threads; };
  if (n <= kFew) {
    constexpr int kTokens = D == 64 ? 16 : 8;
    p.kv_blocks = static_cast<uint32_t>((n + kTokens - 1) / kTokens * p.g.n_kv_heads);
    const dim3 grid(static_cast<unsigned>(p.kv_blocks + q_blocks(1)));
    if (direct)
      hipLaunchKernelGGL((kv4_append_few_kernel<D, XDT, YDT, true>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((kv4_append_few_kernel<D, XDT, YDT, false>), grid, block, 0, stream, p);
    return;
  }
  // (the first tile may begin up to 31 tokens before token 0)
  const int64_t kv = (n + 2 * kKv4Block - 2) / kKv4Block * p.g.n_kv_heads;
  const bool many = q_blocks(kAppendHeads) >= 1024;
  const int64_t total = kv + q_blocks(many ? kAppendHeads : 1);
  // k and v, whose way is longest, go first up to about two fills of the chip (at 71 to
  // 96 registers it holds 1280 to 1792 workgroups); beyond, they are spread over the
  // launch.  Time spread over time first, of 27 cases of 1100 to 8192 tokens: 1.01 to 1.16
  // up to 1134 workgroups, 0.98 to 1.07 (mean 1.03) of 1500 to 2300, 0.99 to 1.04 around
  // 2600, 0.97, 1.04, 0.97 at 2759, 3088, 3447, 0.94 to 0.98 from 4100 on (8192 tokens, D =
  // 128: 30.8 us, 31.8 first; of fp32 44.2, 47.0).  A 32-bit fraction, rounded up, so that
  // each step is 0 or 1 and all are there by the end.
  p.kv_blocks = static_cast<uint32_t>(kv);
  if (total > kAtOnce) p.kv_share = static_cast<uint32_t>(((static_cast<uint64_t>(kv) << 32) + total - 1) / total);
  p.stream = n * p.a.q.heads * D * act_bytes(YDT) > kStreamBytes;
  const dim3 grid(static_cast<unsigned>(total));
  if (many && direct)
    hipLaunchKernelGGL((kv4_append_kernel<D, XDT, YDT, kAppendHeads, true>), grid, block, 0, stream, p);
  else if (many)
    hipLaunchKernelGGL((kv4_append_kernel<D, XDT, YDT, kAppendHeads, false>), grid, block, 0, stream, p);
  else if (direct)
    hipLaunchKernelGGL((kv4_append_kernel<D, XDT, YDT, 1, true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((kv4_append_kernel<D, XDT, YDT, 1, false>), grid, block, 0, stream, p);
}

template <int D, int XDT>
void launch_x(AppendArgs& p, int ydt, hipStream_t stream) {
  if (ydt == kActF32)
    launch_xy<D, XDT, kActF32>(p, stream);
  else if (ydt == kActF16)
    launch_xy<D, XDT, kActF16>(p, stream);
  else
    launch_xy<D, XDT, kActBf16>(p, stream);
}

template <int D>
void launch_d(AppendArgs& p, int xdt, int ydt, hipStream_t stream) {
  if (xdt == kActF32)
    launch_x<D, kActF32>(p, ydt, stream);
  else if (xdt == kActF16)
    launch_x<D, kActF16>(p, ydt, stream);
  else
    launch_x<D, kActBf16>(p, ydt, stream);
}

}  // namespace

hipError_t launch_kv4_append(const Kv4Geom& g, int head_dim, const RopeArgs& a, const Kv4Rows& r, int xdt, int ydt,
                             hipStream_t stream) {
  AppendArgs p{g, a, r, 0, 0, 0};
  if (head_dim == 64)
    launch_d<64>(p, xdt, ydt, stream);
  else
    launch_d<128>(p, xdt, ydt, stream);
  return hipGetLastError();
}

}  // namespace sherry
