// Attention of new tokens over the 4-bit key/value cache.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j,  j <= position of i
//
// One pass over the cache with a running maximum and sum.  A wave takes 16
// rows (tokens x query heads of one key head) and blocks of 32 cached tokens:
//
//   S^T [32 tokens x 16 rows] = K Q^T     v_mfma_f32_16x16x32_f16
//   O^T [D x 16 rows]        += V^T P^T   the same instruction
//
// Transposed, so that a lane's scores (four tokens of each half block, one row)
// are its P^T operand as they stand: the layout of V numbers the tokens of the
// product's reduction axis the way the first product leaves them.
//
// K codes enter the product as fp16 subnormals (code c at bits 0-3 is c 2^-24,
// at bits 4-7 c 2^-20; the queries of those products are scaled by 2^-4), so
// unpacking costs a mask per two codes; with codes c and queries q
//   q . k_j = s_j (q . c_j) + z_j sum(q)      per 64 values
// restores scale and zero point in fp32.  q is scaled to fp16 by a power of two
// per row, exactly for both input types.  V is restored to fp16 in registers
// (1024 + c, - 1024, * s + z: one rounding), so that one P serves all groups.
#include <algorithm>

#include "kv4.h"

namespace sherry {
namespace {

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * kWave;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// P is held times 2^7 (fp16 keeps 2^-14 .. 65504: weights down to 2^-21 of the
// running maximum in full precision), and the running maximum is only raised
// when a score exceeds it by 2^8: P <= 2^15.
constexpr float kPExp = 7.0f;
constexpr float kSlack = 8.0f;
constexpr float kNoMax = -1.0e30f;

template <int D>
struct Stage {  // one block's operands, as loaded
  u32x4_t k[D / 32], v[D / 64], ks[D / 64], kz[D / 64], vs[D / 64], vz[D / 64];
};

template <int D>
__device__ __forceinline__ void load_block(const uint8_t* blk, int lane, Stage<D>& st) {
  using L = Kv4Layout<D>;
  const SHERRY_GLOBAL uint8_t* b = gmem(blk);
  const int g = lane >> 4;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    st.k[i] = *reinterpret_cast<const SHERRY_GLOBAL u32x4_t*>(b + i * 1024 + lane * 16);
    st.v[i] = *reinterpret_cast<const SHERRY_GLOBAL u32x4_t*>(b + L::kVOff + i * 1024 + lane * 16);
    const SHERRY_GLOBAL u32x4_t* p = reinterpret_cast<const SHERRY_GLOBAL u32x4_t*>(b + L::kPOff + i * 256 + g * 16);
    st.ks[i] = p[0], st.kz[i] = p[4], st.vs[i] = p[8], st.vz[i] = p[12];
  }
}

__device__ __forceinline__ half8_t frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4_t w = {a, b, c, d};
  return __builtin_bit_cast(half8_t, w);
}

// fp16 value i of four packed dwords, as fp32
__device__ __forceinline__ float half_of(const u32x4_t& w, int i) {
  const half8_t h = __builtin_bit_cast(half8_t, w);
  return static_cast<float>(h[i]);
}

__device__ __forceinline__ uint32_t restore2(uint32_t biased, half2_t bias, uint32_t s, uint32_t z) {
  half2_t c = __builtin_bit_cast(half2_t, biased) - bias;  // exact
  c = __builtin_elementwise_fma(c, __builtin_bit_cast(half2_t, s), __builtin_bit_cast(half2_t, z));
  return __builtin_bit_cast(uint32_t, c);
}

template <int DT>
__device__ __forceinline__ float half_bits(uint32_t h) {
  return DT == kActF16 ? static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)))
                       : __uint_as_float(h << 16);
}

struct SeqRange {
  int64_t first;  // first token (row of q)
  int32_t n;      // new tokens
  int32_t len;    // cached tokens, new ones included
};

__device__ __forceinline__ SeqRange seq_range(const AttnArgs& a, int s) {
  SeqRange r;
  if (a.cu_q) {
    const int64_t b = min(max(static_cast<int64_t>(gmem(a.cu_q)[s]), int64_t(0)), a.n_tokens);
    const int64_t e = min(max(static_cast<int64_t>(gmem(a.cu_q)[s + 1]), b), a.n_tokens);
    r.first = b;
    r.n = static_cast<int32_t>(e - b);
  } else {
    r.first = static_cast<int64_t>(s) * a.max_q;
    r.n = a.max_q;
  }
  const int64_t cap = static_cast<int64_t>(a.table_width) << a.c.page_shift;
  r.len = static_cast<int32_t>(min(static_cast<int64_t>(max(gmem(a.kv_lens)[s], 0)), cap));
  return r;
}

// Rows of a sequence and key head: row r is token r / group, query head
// r % group of the key head's group.
template <int D, int DT>
__global__ __launch_bounds__(kAttnThreads) void kv4_attn_kernel(AttnArgs a) {
  constexpr int NG = D / 64;   // scale groups
  constexpr int KS = D / 32;   // products along D per 16 tokens
  constexpr int NT = D / 16;   // 16-value tiles of the output
  constexpr int kPad = D + 4;  // LDS row stride: 16 rows start 4 banks apart
  __shared__ float lds_o[kAttnWaves][16][kPad];
  __shared__ float lds_m[kAttnWaves][16], lds_l[kAttnWaves][16];

  const int split = static_cast<int>(blockIdx.x % a.splits);
  const int st_id = static_cast<int>(blockIdx.x / a.splits);
  const int seq = st_id / a.row_tiles;
  const int tile = st_id - seq * a.row_tiles;
  const int kvh = blockIdx.y;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & (kWave - 1);
  const int col = lane & 15, g = lane >> 4;
  const SeqRange sr = seq_range(a, seq);
  const int n = min(sr.n, a.max_q);
  const int rows = n * a.group;
  const int row0 = tile * 16;
  if (row0 >= rows) return;
  const int nrow = min(16, rows - row0);

  // visible tokens: row r sees tokens below lim(r)
  const int lim_lo = max(sr.len - sr.n + row0 / a.group + 1, 0);
  const int lim_hi = max(min(sr.len - sr.n + (row0 + nrow - 1) / a.group + 1, sr.len), 0);
  const int row = min(row0 + col, rows - 1);
  const int tok = row / a.group;
  const int head = kvh * a.group + (row - tok * a.group);
  const int lim = sr.len - sr.n + tok + 1;

  // the lane's queries: values 32 ks + 8 g .. + 7 of its row, scaled to fp16
  half8_t q[KS];
  float sumq[NG];
  float kc;  // score scale
  {
    float f[KS][8];
    float amax = 0.0f;
    const int64_t at = (sr.first + tok) * a.q_st + head * a.q_sh + 8 * g;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      load8<DT>(a.q, at + 32 * i, f[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[i][j]));
    }
    amax = fmaxf(amax, __shfl_xor(amax, 16));
    amax = fmaxf(amax, __shfl_xor(amax, 32));
    const int e = max(static_cast<int>(__float_as_uint(amax) >> 23), 1) - 127;
    const float unit = a.scale * kLog2e;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += f[2 * i][j] + f[2 * i + 1][j];
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      sumq[i] = s * unit;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        q[i][j] = static_cast<_Float16>(__builtin_ldexpf(f[i][j], 11 - e - 4 * (i & 1)));
    kc = __builtin_ldexpf(unit, 24 + e - 11);
  }

  f32x4_t o[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i] = f32x4_t{0, 0, 0, 0};
  float m = kNoMax, l = 0.0f;

  // this workgroup's blocks, taken by its waves in turn
  const int nblk = (lim_hi + kKv4Block - 1) / kKv4Block;
  const int per = (nblk + a.splits - 1) / a.splits;
  const int b_end = min(nblk, (split + 1) * per);
  const int page_blocks = a.c.page_shift - 5;
  const int32_t* table = a.table + static_cast<int64_t>(seq) * a.table_stride;
  for (int b = split * per + wave; b < b_end; b += kAttnWaves) {
    const int64_t page = gmem(table)[b >> page_blocks];
    if (page < 0 || page >= a.c.n_pages) continue;  // no such page: no such tokens
    Stage<D> st;
    load_block<D>(a.c.data + kv4_block_off<D>(a.c, page, kvh, b & ((1 << page_blocks) - 1)), lane, st);

    f32x4_t acc[2][NG];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const uint32_t w0 = D == 64 ? st.k[0][2 * t] : st.k[t][2 * i];
        const uint32_t w1 = D == 64 ? st.k[0][2 * t + 1] : st.k[t][2 * i + 1];
        const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
        constexpr uint32_t kLo = 0x000F000Fu, kHi = 0x00F000F0u;
        f32x4_t c = {0, 0, 0, 0};
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(frag(w0 & kLo, h0 & kLo, w1 & kLo, h1 & kLo), q[2 * i], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(frag(w0 & kHi, h0 & kHi, w1 & kHi, h1 & kHi), q[2 * i + 1], c, 0, 0, 0);
        acc[t][i] = c;
      }

    const int t0 = b * kKv4Block + 4 * g;  // the lane's tokens: t0 + i, t0 + 16 + i
    const bool edge = (b + 1) * kKv4Block > lim_lo;
    if (edge) {
      // tokens past the sequence may hold anything: their V must be finite
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t keep = t0 + 16 * (i >> 2) + (i & 3) < sr.len ? 0xFFFFu << (16 * (i & 1)) : 0u;
        const uint32_t mask = keep | ~(0xFFFFu << (16 * (i & 1)));
#pragma unroll
        for (int k = 0; k < NG; ++k) st.vs[k][i >> 1] &= mask, st.vz[k][i >> 1] &= mask;
      }
    }
    // x = score - m in powers of two
    float x[8];
    auto scores = [&](float mm) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float s = half_of(st.ks[0], i) * acc[i >> 2][0][i & 3];
        float u = __builtin_fmaf(half_of(st.kz[0], i), sumq[0], -mm);
        if constexpr (NG == 2) {
          s = __builtin_fmaf(half_of(st.ks[1], i), acc[i >> 2][1][i & 3], s);
          u = __builtin_fmaf(half_of(st.kz[1], i), sumq[1], u);
        }
        x[i] = __builtin_fmaf(s, kc, u);
      }
      if (edge) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = t0 + 16 * (i >> 2) + (i & 3) < lim ? x[i] : -__builtin_inff();
      }
    };
    auto top = [&]() {
      return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    };
    scores(m - kPExp);
    if (__any(top() > kPExp + kSlack)) {
      scores(0.0f);
      float mx = top();
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float m_new = fmaxf(m, mx);
      const float alpha = __builtin_amdgcn_exp2f(m - m_new);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i] *= alpha;
      scores(m - kPExp);
    }
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(x[i]);
      l += p[i];
    }
    const half8_t pf = frag(pack2<kActF16>(p[0], p[1]), pack2<kActF16>(p[2], p[3]), pack2<kActF16>(p[4], p[5]),
                            pack2<kActF16>(p[6], p[7]));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      constexpr half2_t k1024 = {static_cast<_Float16>(1024.0f), static_cast<_Float16>(1024.0f)};
      constexpr half2_t k64 = {static_cast<_Float16>(64.0f), static_cast<_Float16>(64.0f)};
      const u32x4_t vs = st.vs[i >> 1], vz = st.vz[i >> 1];
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t w = st.v[i >> 1][2 * (i & 1) + t], h = w >> 8;
        lo[2 * t] = restore2((w & 0x000F000Fu) | 0x64006400u, k1024, vs[2 * t], vz[2 * t]);
        lo[2 * t + 1] = restore2((h & 0x000F000Fu) | 0x64006400u, k1024, vs[2 * t + 1], vz[2 * t + 1]);
        hi[2 * t] = restore2((w & 0x00F000F0u) | 0x54005400u, k64, vs[2 * t], vz[2 * t]);
        hi[2 * t + 1] = restore2((h & 0x00F000F0u) | 0x54005400u, k64, vs[2 * t + 1], vz[2 * t + 1]);
      }
      o[2 * i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(frag(lo[0], lo[1], lo[2], lo[3]), pf, o[2 * i], 0, 0, 0);
      o[2 * i + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(frag(hi[0], hi[1], hi[2], hi[3]), pf, o[2 * i + 1], 0, 0, 0);
    }
  }

  // join the waves: every wave's rows on a common maximum
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (col < nrow) {
    if (g == 0) lds_m[wave][col] = m, lds_l[wave][col] = l;
#pragma unroll
    for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4_t*>(&lds_o[wave][col][16 * i + 4 * g]) = o[i];
  }
  __syncthreads();
  for (int u = threadIdx.x; u < nrow * (D / 4); u += kAttnThreads) {
    const int r = u / (D / 4), d = 4 * (u % (D / 4));
    float mm = lds_m[0][r];
#pragma unroll
    for (int w = 1; w < kAttnWaves; ++w) mm = fmaxf(mm, lds_m[w][r]);
    float ll = 0.0f;
    f32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(lds_m[w][r] - mm);
      ll = __builtin_fmaf(f, lds_l[w][r], ll);
      const f32x4_t t = *reinterpret_cast<const f32x4_t*>(&lds_o[w][r][d]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(f, t[j], v[j]);
    }
    const int rr = row0 + r;
    const int ti = rr / a.group;
    const int64_t token = sr.first + ti;
    const int hd = kvh * a.group + (rr - ti * a.group);
    if (a.splits > 1) {
      const int64_t at = (static_cast<int64_t>(split) * a.n_tokens + token) * a.n_q_heads + hd;
      *gmem(reinterpret_cast<f32x4_t*>(a.part_o + at * D + d)) = v;
      if (d == 0) *gmem(reinterpret_cast<f32x2_t*>(a.part_ml + at * 2)) = f32x2_t{mm, ll};
    } else {
      const float inv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : ll);
      u32x2_t out = {pack2<DT>(v[0] * inv, v[1] * inv), pack2<DT>(v[2] * inv, v[3] * inv)};
      *gmem(reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + token * a.o_st + hd * a.o_sh + d)) = out;
      if (a.lse && d == 0)
        gmem(a.lse)[token * a.n_q_heads + hd] =
            ll == 0.0f ? -__builtin_inff() : (mm - kPExp + __builtin_log2f(ll)) * kLn2;
    }
  }
}

// Joins the splits of every row: a quarter of a wave (D = 64) or half of one
// (D = 128) per row, four values a lane, splits in their order.
template <int D, int DT>
__global__ __launch_bounds__(kAttnThreads) void kv4_join_kernel(AttnArgs a) {
  constexpr int kLanes = D / 4;
  const int seq = static_cast<int>(blockIdx.x / a.join_blocks);
  const SeqRange sr = seq_range(a, seq);
  const int n = min(sr.n, a.max_q);
  const int64_t u =
      (static_cast<int64_t>(blockIdx.x % a.join_blocks) * kAttnThreads + threadIdx.x) / kLanes;
  const int d = 4 * (threadIdx.x % kLanes);
  const int64_t ti = u / a.n_q_heads;
  if (ti >= n) return;
  const int hd = static_cast<int>(u - ti * a.n_q_heads);
  const int64_t token = sr.first + ti;
  const int64_t at = token * a.n_q_heads + hd, step = a.n_tokens * a.n_q_heads;
  float m = kNoMax, l = 0.0f;
  f32x4_t v = {0, 0, 0, 0};
  for (int s = 0; s < a.splits; ++s) {
    const f32x2_t ml = *gmem(reinterpret_cast<const f32x2_t*>(a.part_ml + (at + s * step) * 2));
    const f32x4_t t = *gmem(reinterpret_cast<const f32x4_t*>(a.part_o + (at + s * step) * D + d));
    const float m_new = fmaxf(m, ml.x);
    const float f0 = __builtin_amdgcn_exp2f(m - m_new), f1 = __builtin_amdgcn_exp2f(ml.x - m_new);
    m = m_new;
    l = __builtin_fmaf(f1, ml.y, l * f0);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(f1, t[j], v[j] * f0);
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
  u32x2_t out = {pack2<DT>(v[0] * inv, v[1] * inv), pack2<DT>(v[2] * inv, v[3] * inv)};
  *gmem(reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + token * a.o_st + hd * a.o_sh + d)) = out;
  if (a.lse && d == 0)
    gmem(a.lse)[at] = l == 0.0f ? -__builtin_inff() : (m - kPExp + __builtin_log2f(l)) * kLn2;
}

template <int D, int DT>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.splits) * a.n_seqs * a.row_tiles),
                  static_cast<unsigned>(a.c.n_kv_heads));
  hipLaunchKernelGGL((kv4_attn_kernel<D, DT>), grid, dim3(kAttnThreads), 0, stream, a);
  if (a.splits > 1) {
    AttnArgs j = a;
    j.join_blocks = static_cast<int32_t>(
        (static_cast<int64_t>(a.max_q) * a.n_q_heads * (D / 4) + kAttnThreads - 1) / kAttnThreads);
    const dim3 jg(static_cast<unsigned>(static_cast<int64_t>(j.join_blocks) * a.n_seqs));
    hipLaunchKernelGGL((kv4_join_kernel<D, DT>), jg, dim3(kAttnThreads), 0, stream, j);
  }
  return hipGetLastError();
}

}  // namespace

// Splits of the cached tokens: enough workgroups to fill the chip, each with
// at least two blocks per wave.
int32_t kv4_attn_splits(int64_t workgroups, int64_t max_kv) {
  constexpr int64_t kWant = 1024;
  const int64_t blocks = (max_kv + kKv4Block - 1) / kKv4Block;
  const int64_t most = (blocks + 2 * kAttnWaves - 1) / (2 * kAttnWaves);
  const int64_t want = (kWant + workgroups - 1) / workgroups;
  return static_cast<int32_t>(std::max<int64_t>(1, std::min(most, want)));
}

hipError_t launch_kv4_attn(const AttnArgs& a, int head_dim, int dt, hipStream_t stream) {
  if (head_dim == 64) return dt == kActF16 ? launch_d<64, kActF16>(a, stream) : launch_d<64, kActBf16>(a, stream);
  return dt == kActF16 ? launch_d<128, kActF16>(a, stream) : launch_d<128, kActBf16>(a, stream);
}

}  // namespace sherry
