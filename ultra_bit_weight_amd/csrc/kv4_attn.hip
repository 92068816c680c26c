// Attention of new tokens over the 4-bit key/value cache.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j,  j <= position of i
//
// One pass over the cache with a running maximum and sum, on blocks of 32
// cached tokens and tiles of 16 rows (tokens x query heads of one key head):
//
//   S^T [32 tokens x 16 rows] = K Q^T     v_mfma_f32_16x16x32_f16
//   O^T [D x 16 rows]        += V^T P^T   the same instruction
//
// Transposed, so that a lane's scores (four tokens of each half block, one row)
// are its P^T operand as they stand: the layout of V numbers the tokens of the
// product's reduction axis the way the first product leaves them.
//
// Scale and zero point stay outside the products, whose operands are the codes
// themselves (exact in 16 bits) on one side.  Per 64 values, with codes c:
//   q . k_j = s_j (q . c_j) + z_j sum(q)
//   sum_j p_j v_j = sum_j P_j (c_j - mid) + sum_j p_j (z_j + mid s_j),  P = p s
// So K enters without rounding, and q as it is where rows are many; where they
// are few it is brought to fp16 by a power of two for each row, which rounds
// what lies below 2^-25 of the row's largest to 2^-36 of that.  The one rounding
// inside is P to fp16: 2^-11 of each term (2^-32 of the row's largest P where
// that is more), like an fp16 result's own, an eighth of a bf16 one's.
// mid = 7.5 centres V's codes: sums of 0..15 would cancel against the zero
// point's part to a result that over a long axis is hundreds of times smaller.
//
// Of P's rounding error, where results are fp16 and rows few, a second operand
// is made and multiplied too, which leaves the result's own rounding alone
// (measured against 64 bits, of the norm: 0.00021, and 0.00031 without it; that
// costs 3 % of one token over 131072).  With more rows the products are the
// work, and it would be 30 % of a 2048-token chunk: 0.00031 stays there.
//
// Unpacking.  The matrix core aligns a product by its operands' exponent fields
// and cuts off what falls below, so a subnormal operand with k leading zeros
// costs k bits of its sums.  V's codes (a mask) are made normal by the fma that
// centres them.  K's, where rows are few, take a shift and a mask, to bits 4-7: 3
// to 6 leading zeros keep the scores to 2e-7 of their size (7 to 10 of them, in
// bits 0-3, to 2e-6; normal numbers by an fma: the same 2e-7, but 7 % of a
// batch's time).  Where rows are many they are 16 + c, whose four bits lie behind
// an exponent in fp16 as in bf16 (a shift and one mask-and-or), with 16 s taken
// off z.  The powers of two are taken off the scores and off O.
#include <algorithm>
#include <type_traits>

#include "kv4.h"

namespace sherry {
namespace {

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * kWave;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum is one of score + log2(V scale), so that P's largest is
// 2^kPExp when it is set; it is raised again only when some P passes kPTop
// (fp16 ends at 65504).  P keeps full precision down to 2^-21 of the largest.
// A V scale of 0 (a constant group, a token never written) hides p from P: it
// counts as 2^-24 for the maximum, and the sum of p is watched too.
// What is kept as the maximum m is what is subtracted: kPExp less, rounded.
constexpr float kPExp = 7.0f;
constexpr float kPTop = 32768.0f;
constexpr float kSumTop = 1.0e18f;
constexpr float kNoMax = -3.0e38f;  // below every score
constexpr float kMid = 7.5f;        // centre of the codes
constexpr uint32_t kLoMask = 0x000F000Fu, kHiMask = 0x00F000F0u;

__device__ __forceinline__ half8_t frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4_t w = {a, b, c, d};
  return __builtin_bit_cast(half8_t, w);
}

__device__ __forceinline__ f32x4_t mfma(half8_t a, half8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// V's operands: (code - kMid) 2^-10 from bits 0-3 of each half, 2^-6 from bits
// 4-7, exact.
template <bool kHigh>
__device__ __forceinline__ uint32_t v_pair(uint32_t w) {
  constexpr _Float16 up = 16384.0f16, off = kHigh ? -kMid / 64 : -kMid / 1024;
  const half2_t c = __builtin_bit_cast(half2_t, w & (kHigh ? kHiMask : kLoMask));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c, half2_t{up, up}, half2_t{off, off}));
}
template <bool kHigh>
__device__ __forceinline__ half8_t v_operand(uint32_t w0, uint32_t w1) {
  return frag(v_pair<kHigh>(w0), v_pair<kHigh>(w0 >> 8), v_pair<kHigh>(w1), v_pair<kHigh>(w1 >> 8));
}
// K's operands of few rows: codes in bits 4-7, fp16 subnormals of 2^-20.
template <bool kHigh>
__device__ __forceinline__ half8_t k_operand(uint32_t w0, uint32_t w1) {
  if (kHigh) return frag(w0 & kHiMask, (w0 >> 8) & kHiMask, w1 & kHiMask, (w1 >> 8) & kHiMask);
  return frag((w0 << 4) & kHiMask, (w0 >> 4) & kHiMask, (w1 << 4) & kHiMask, (w1 >> 4) & kHiMask);
}

// K's operands of many rows: 16 + code, in the queries' own type.  So q enters as
// it is, and rows of any sizes share a workgroup: fp16 for both types needs powers
// of two for bf16, and one for each row costs a factor a score (2048 tokens over
// 8192 221 us against 213, ragged prompts 114.7 against 112.1).
constexpr float kBase = 16.0f;
template <int DT, bool kHigh>
__device__ __forceinline__ u32x4_t k_plus_base(uint32_t w0, uint32_t w1) {
  constexpr bool kF16 = DT == kActF16;
  // the code at the mantissa's top, bits 6-9 or 3-6 of a half, behind the exponent of 16
  constexpr uint32_t mask = kF16 ? 0x03C003C0u : 0x00780078u, base = kF16 ? 0x4C004C00u : 0x41804180u;
  auto at = [](uint32_t w, int from) {  // the code that starts at bit `from` of a half
    const int left = (kF16 ? 6 : 3) - from;
    return ((left >= 0 ? w << (left & 31) : w >> (-left & 31)) & mask) | base;
  };
  constexpr int lo = kHigh ? 4 : 0;
  return u32x4_t{at(w0, lo), at(w0, lo + 8), at(w1, lo), at(w1, lo + 8)};
}
template <int DT>
__device__ __forceinline__ f32x4_t mfma_k(u32x4_t k, u32x4_t q, f32x4_t c) {
  typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
  if constexpr (DT == kActF16) return mfma(__builtin_bit_cast(half8_t, k), __builtin_bit_cast(half8_t, q), c);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8_t, k), __builtin_bit_cast(bf8_t, q), c, 0, 0, 0);
}

// fp16 value i of four packed dwords, as fp32
__device__ __forceinline__ float half_of(const u32x4_t& w, int i) {
  return static_cast<float>(__builtin_bit_cast(half8_t, w)[i]);
}

struct SeqRange {
  int64_t first;  // first token (row of q)
  int32_t n;      // new tokens
  int32_t len;    // cached tokens, new ones included
};

// New tokens only (len 0).  (Loads before any branch, so that they and the
// lengths' go out together.)
__device__ __forceinline__ SeqRange new_range(const AttnArgs& a, int s) {
  const SHERRY_GLOBAL int32_t* cu = gmem(a.cu_q ? a.cu_q : a.kv_lens);
  const int64_t from = cu[s], to = cu[a.cu_q ? s + 1 : s];
  const int64_t b = min(max(from, int64_t(0)), a.n_tokens);
  const int64_t e = min(max(to, b), a.n_tokens);
  return a.cu_q ? SeqRange{b, static_cast<int32_t>(e - b), 0}
                : SeqRange{static_cast<int64_t>(s) * a.max_q, a.max_q, 0};
}

__device__ __forceinline__ SeqRange seq_range(const AttnArgs& a, int s) {
  const int32_t len = gmem(a.kv_lens)[s];
  SeqRange r = new_range(a, s);
  const int64_t cap = static_cast<int64_t>(a.table_width) << a.c.page_shift;
  r.len = static_cast<int32_t>(min(static_cast<int64_t>(max(len, 0)), cap));
  return r;
}

// A workgroup's share of the call.  Key heads vary fastest (with 8 of them, each
// XCD keeps one head's blocks in its L2), then splits, sequences, and row tiles
// from the last: the last rows see most tokens, and start first.
struct Place {
  int tile, seq, split, head;
};
__device__ __forceinline__ Place place(const AttnArgs& a) {
  Place p;
  int i = static_cast<int>(blockIdx.x);
  const int by_head = a.by_kv_heads(i);
  p.head = i - by_head * a.c.n_kv_heads;
  i = a.by_splits(by_head);
  p.split = by_head - i * a.splits;
  const int back = a.by_seqs(i);
  p.seq = i - back * a.n_seqs;
  p.tile = a.row_tiles - 1 - back;
  return p;
}

// Codes of one block as a lane loads them.
template <int D>
struct KCodes {
  u32x4_t w[D / 64];
  // dword pair of half block t, scale group gr: values 64 gr .. 64 gr + 63
  __device__ __forceinline__ u32x2_t pair(int t, int gr) const {
    return D == 64 ? u32x2_t{w[0][2 * t], w[0][2 * t + 1]} : u32x2_t{w[t][2 * gr], w[t][2 * gr + 1]};
  }
};
template <int D>
struct VCodes {
  u32x4_t w[D / 64];
  // dword pair of values 32 i .. 32 i + 31
  __device__ __forceinline__ u32x2_t pair(int i) const { return {w[i >> 1][2 * (i & 1)], w[i >> 1][2 * (i & 1) + 1]}; }
};
// Scales and zero points of the lane's eight tokens (fp16).
template <int D>
struct Params {
  u32x4_t ks[D / 64], kz[D / 64], vs[D / 64], vz[D / 64];
};

template <int D>
__device__ __forceinline__ void load_k(const uint8_t* blk, int lane, KCodes<D>& k) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    k.w[i] = *reinterpret_cast<const SHERRY_GLOBAL u32x4_t*>(gmem(blk) + i * 1024 + lane * 16);
}
template <int D>
__device__ __forceinline__ void load_v(const uint8_t* blk, int lane, VCodes<D>& v) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    v.w[i] =
        *reinterpret_cast<const SHERRY_GLOBAL u32x4_t*>(gmem(blk) + Kv4Layout<D>::kVOff + i * 1024 + lane * 16);
}
template <int D>
__device__ __forceinline__ void load_p(const uint8_t* blk, int g, Params<D>& p) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const SHERRY_GLOBAL u32x4_t* s =
        reinterpret_cast<const SHERRY_GLOBAL u32x4_t*>(gmem(blk) + Kv4Layout<D>::kPOff + i * 256 + g * 16);
    p.ks[i] = s[0], p.kz[i] = s[4], p.vs[i] = s[8], p.vz[i] = s[12];
  }
}

// Zeroes the scales of tokens that lie past `len` (their bytes may be anything,
// and 0 * NaN is not 0); t0 is the lane's first token.
template <int D>
__device__ __forceinline__ Params<D> drop_tail(Params<D> p, int t0, int len) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + 16 * (i >> 1) + 2 * (i & 1);
    const uint32_t mask = (t < len ? 0xFFFFu : 0u) | (t + 1 < len ? 0xFFFF0000u : 0u);
#pragma unroll
    for (int k = 0; k < D / 64; ++k) p.ks[k][i] &= mask, p.kz[k][i] &= mask, p.vs[k][i] &= mask, p.vz[k][i] &= mask;
  }
  return p;
}

// A lane's queries, values 32 i + 8 g .. + 7 of one row.
template <int D, int DT>
struct Queries {
  float f[D / 32][8];
  __device__ __forceinline__ void load(const void* q, int64_t at) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) load8<DT>(q, at + 32 * i, f[i]);
  }
  // largest magnitude of the row, 0 if that is infinite
  __device__ __forceinline__ float top() const {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[i][j]));
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    return m < __builtin_inff() ? m : 0.0f;
  }
  // sum of each scale group, times unit
  __device__ __forceinline__ void sums(float unit, float (&sumq)[D / 64]) const {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += f[2 * i][j] + f[2 * i + 1][j];
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      sumq[i] = s * unit;
    }
  }
  // as they came
  __device__ __forceinline__ u32x4_t bits(int i) const {
    return u32x4_t{pack2<DT>(f[i][0], f[i][1]), pack2<DT>(f[i][2], f[i][3]), pack2<DT>(f[i][4], f[i][5]),
                   pack2<DT>(f[i][6], f[i][7])};
  }
  // fp16 operands, the row's largest at 2^11
  __device__ __forceinline__ void operands(int e, half8_t (&q)[D / 32]) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) q[i][j] = static_cast<_Float16>(__builtin_ldexpf(f[i][j], 11 - e));
  }
};

__device__ __forceinline__ int exponent_of(float v) { return max(static_cast<int>(__float_as_uint(v) >> 23), 1) - 127; }

// Running state of one tile of 16 rows: O^T (without the zero-point part), the
// zero-point part, maximum and sum.
template <int D>
struct Acc {
  f32x4_t o[D / 16];
  float w[D / 64];
  float m, l;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < D / 64; ++i) w[i] = 0.0f;
    m = kNoMax, l = 0.0f;
  }
  __device__ __forceinline__ void scale(float f) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] *= f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) w[i] *= f;
    l *= f;
  }
  // value i of tile nt: odd tiles are made of high nibbles
  __device__ __forceinline__ float value(int nt, int i) const {
    return __builtin_fmaf(o[nt][i], nt & 1 ? 64.0f : 1024.0f, w[nt >> 2]);
  }
  // after the last block: sums over the four lane groups of a row
  __device__ __forceinline__ void finish() {
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      w[i] += __shfl_xor(w[i], 16);
      w[i] += __shfl_xor(w[i], 32);
    }
  }
};

// The lane's eight tokens' parameters of group k: K scale and zero point, V scale,
// and V zero point + kMid V scale.
template <int D>
struct RawParams {  // made from fp16 as they are used
  const Params<D>& p;
  float unit;  // of the products, sums of q included, in powers of two of the softmax
  __device__ __forceinline__ float ks(int k, int i) const { return half_of(p.ks[k], i); }
  __device__ __forceinline__ float kz(int k, int i) const { return half_of(p.kz[k], i); }
  __device__ __forceinline__ float vs(int k, int i) const { return half_of(p.vs[k], i); }
  __device__ __forceinline__ float vz(int k, int i) const {
    return __builtin_fmaf(half_of(p.vs[k], i), kMid, half_of(p.vz[k], i));
  }
};
template <int D>
struct LdsParams {  // ready-made, in LDS (at the lane group's eight tokens), the unit in K's scale
  const float* at;
  __device__ __forceinline__ float ks(int k, int i) const { return at[(4 * k) * kKv4Block + i]; }
  __device__ __forceinline__ float kz(int k, int i) const { return at[(4 * k + 1) * kKv4Block + i]; }
  __device__ __forceinline__ float vs(int k, int i) const { return at[(4 * k + 2) * kKv4Block + i]; }
  __device__ __forceinline__ float vz(int k, int i) const { return at[(4 * k + 3) * kKv4Block + i]; }
};

// The softmax step of one tile: scores from the products c (S^T of each scale
// group) to P operands, one per group.  kEdge: tokens from lim on are not seen
// (t0 is the lane's first token).
template <int D, bool kEdge, bool kTwo, class P>
__device__ __forceinline__ void softmax_step(Acc<D>& a, const f32x4_t (&c)[2][D / 64], const P& pr,
                                             const float (&sumq)[D / 64], int t0, int lim,
                                             half8_t (&pf)[kTwo ? 2 : 1][D / 64]) {
  constexpr int NG = D / 64;
  constexpr bool kReady = std::is_same_v<P, LdsParams<D>>;  // the unit is in the parameters
  float p[8], ps[NG][8], top, sum;
  // The maximum is taken off the rounded score that it was taken of.  Folded into
  // the first fma it would round apart from that, by units from scores (or parts
  // of scores) of 2^24 on, and the largest weight be infinite or 0; the operation
  // costs 219 us against 213 for 2048 tokens over 8192, 113.1 against 112.0 for
  // ragged prompts, and where rows are few 1 % at most (12.2 against 12.0 for one
  // token over 40000; 21.2 and 82.8 for 131072 and a batch as before).
  auto score = [&](int i, float m) {
    float u = pr.kz(0, i) * sumq[0];
#pragma unroll
    for (int k = 1; k < NG; ++k) u = __builtin_fmaf(pr.kz(k, i), sumq[k], u);
#pragma unroll
    for (int k = 0; k < NG; ++k) u = __builtin_fmaf(pr.ks(k, i), c[i >> 2][k][i & 3], u);
    if constexpr (!kReady) u *= pr.unit;
    u -= m;
    if constexpr (kEdge) u = t0 + 16 * (i >> 2) + (i & 3) < lim ? u : -__builtin_inff();
    return u;
  };
  auto weights = [&]() {
    top = 0.0f, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(score(i, a.m));
      sum += p[i];
    }
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ps[k][i] = __builtin_fmaf(p[i], pr.vs(k, i), 0.0f);  // (fma: a mixed-precision instruction for fp16)
        top = fmaxf(top, ps[k][i]);
      }
  };
  weights();
  if (__builtin_expect(__any(top > kPTop || sum > kSumTop), 0)) {
    float mx = kNoMax;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = 5.9604644775390625e-8f;  // 2^-24
#pragma unroll
      for (int k = 0; k < NG; ++k) v = fmaxf(v, pr.vs(k, i));
      mx = fmaxf(mx, score(i, 0.0f) + __builtin_amdgcn_logf(v));  // log2
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float m_new = fmaxf(a.m, mx - kPExp);
    a.scale(__builtin_amdgcn_exp2f(a.m - m_new));
    a.m = m_new;
    weights();
  }
  a.l += sum;
#pragma unroll
  for (int k = 0; k < NG; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a.w[k] = __builtin_fmaf(p[i], pr.vz(k, i), a.w[k]);
    pf[0][k] = frag(pack2<kActF16>(ps[k][0], ps[k][1]), pack2<kActF16>(ps[k][2], ps[k][3]),
                    pack2<kActF16>(ps[k][4], ps[k][5]), pack2<kActF16>(ps[k][6], ps[k][7]));
    if constexpr (kTwo) {  // (fma again: one mixed-precision instruction)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        pf[1][k][i] = static_cast<_Float16>(__builtin_fmaf(p[i], pr.vs(k, i), -static_cast<float>(pf[0][k][i])));
    }
  }
}

// Stores of a row's result, four values d .. d + 3: the final one, or a split's
// share.
template <int D, int DT>
__device__ __forceinline__ void store_row(const AttnArgs& a, int split, int64_t token, int head, int d,
                                          const float (&v)[4], float m, float l) {
  if (a.splits > 1) {
    const int64_t at = (static_cast<int64_t>(split) * a.n_tokens + token) * a.n_q_heads + head;
    *gmem(reinterpret_cast<f32x4_t*>(a.part_o + at * D + d)) = f32x4_t{v[0], v[1], v[2], v[3]};
    if (d == 0) *gmem(reinterpret_cast<f32x2_t*>(a.part_ml + at * 2)) = f32x2_t{m, l};
  } else {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const u32x2_t out = {pack2<DT>(v[0] * inv, v[1] * inv), pack2<DT>(v[2] * inv, v[3] * inv)};
    *gmem(reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + token * a.o_st + head * a.o_sh + d)) = out;
    if (a.lse && d == 0)
      gmem(a.lse)[token * a.n_q_heads + head] =
          l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
  }
}

// ---- up to 16 rows: the cached tokens are what there is to share out ----
//
// The workgroup's waves take chunks of G blocks in turn.  With at most 16 / G
// rows, the 16 columns of a tile hold the rows G times over, and the columns of
// copy b are given to block b of the chunk: the products of the G blocks add
// into one S^T, each with the queries zeroed outside its columns, so one
// softmax step serves G blocks.  The copies are separate softmaxes, joined with
// the waves' at the end.  (Rows <= 8, G = 2 against G = 1: 20.7 against 22.8 us
// for one token over 131072, 82.7 against 91.3 for a batch of 48; 4.9 against
// 4.7 for one over 200, where there is little to share.  G = 4 for rows <= 4
// costs more registers than it saves: 26 and 107 us when G = 2 took 22.4 and 90.)
//
// K of the next chunk is loaded as soon as this one's has been multiplied, V
// and the scales likewise, so loads are in flight during the softmax and the
// other product; the page numbers are read a chunk ahead of that.  After the
// last chunk the loads repeat it (from L2): a branch around them would make the
// compiler wait for them where it joins.
template <int D, int DT, int G>
__global__ __launch_bounds__(kAttnThreads, 2) void kv4_attn_few_kernel(AttnArgs a) {
  constexpr int NG = D / 64, KS = D / 32, NT = D / 16;
  constexpr int kRows = 16 / G;
  constexpr bool kTwo = DT == kActF16;  // P's rounding error as a second operand
  constexpr int kParts = kTwo ? 2 : 1;
  constexpr int kPad = D + 4;  // LDS row stride: 16 rows start 4 banks apart
  __shared__ float lds_o[kAttnWaves][16][kPad];
  __shared__ float lds_m[kAttnWaves][16], lds_l[kAttnWaves][16];

  const Place at_place = place(a);
  const int split = at_place.split, seq = at_place.seq, kvh = at_place.head;
  const int row0 = at_place.tile * kRows;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & (kWave - 1);
  const int col = lane & 15, g = lane >> 4;
  const int copy = col / kRows;
  const SeqRange sr = seq_range(a, seq);
  const int rows = min(sr.n, a.max_q) * a.group;
  if (row0 >= rows) return;
  const int nrow = min(kRows, rows - row0);

  // row r sees tokens below lim(r)
  const int lim_lo = max(sr.len - sr.n + a.by_group(row0) + 1, 0);
  const int lim_hi = max(min(sr.len - sr.n + a.by_group(row0 + nrow - 1) + 1, sr.len), 0);
  const int row = min(row0 + col % kRows, rows - 1);
  const int tok = a.by_group(row);
  const int head = kvh * a.group + (row - tok * a.group);
  const int lim = sr.len - sr.n + tok + 1;

  const int nblk = (lim_hi + kKv4Block - 1) / kKv4Block;
  const int chunks = (nblk + G - 1) / G;
  const int per = (chunks + a.splits - 1) / a.splits;
  const int c_end = min(chunks, (split + 1) * per);
  const int c_begin = split * per + wave;
  const int page_blocks = a.c.page_shift - 5;
  const SHERRY_GLOBAL int32_t* table = gmem(a.table) + static_cast<int64_t>(seq) * a.table_stride;

  struct Chunk {
    const uint8_t* at[G];  // its blocks; one that is not there reads the cache's first
    const uint8_t* mine;   // the block of the lane's copy
    bool mine_there, all_there;
  };
  auto pages = [&](int ch, int32_t (&pg)[G]) {
#pragma unroll
    for (int b = 0; b < G; ++b) pg[b] = table[min(ch * G + b, nblk - 1) >> page_blocks];
  };
  auto chunk = [&](int ch, const int32_t (&pg)[G]) {
    Chunk c;
    c.all_there = true;
#pragma unroll
    for (int b = 0; b < G; ++b) {
      const int blk = ch * G + b;
      const bool there = blk < nblk && pg[b] >= 0 && pg[b] < a.c.n_pages;
      const int64_t off = kv4_block_off<D>(a.c, there ? pg[b] : 0, kvh, blk & ((1 << page_blocks) - 1));
      const uint8_t* at = a.c.data + (there ? off : 0);
      c.at[b] = at;
      c.mine = b == 0 || copy == b ? at : c.mine;
      c.mine_there = b == 0 || copy == b ? there : c.mine_there;
      c.all_there = c.all_there && there;
    }
    return c;
  };
  KCodes<D> k[G];
  VCodes<D> v[G];
  Params<D> pr;
  Chunk now, next;
  int32_t pg[G];
  const bool any = c_begin < c_end;
  if (any) {
    pages(c_begin, pg);
    now = chunk(c_begin, pg);
#pragma unroll
    for (int b = 0; b < G; ++b) load_k<D>(now.at[b], lane, k[b]);
    load_p<D>(now.mine, g, pr);
#pragma unroll
    for (int b = 0; b < G; ++b) load_v<D>(now.at[b], lane, v[b]);
    pages(min(c_begin + kAttnWaves, c_end - 1), pg);
  }

  half8_t q[G][KS];
  float sumq[NG];
  float unit;
  {
    Queries<D, DT> f;
    f.load(a.q, (sr.first + tok) * a.q_st + head * a.q_sh + 8 * g);
    const int e = exponent_of(f.top());
    f.sums(__builtin_ldexpf(1.0f, 11 - e - 20), sumq);  // in the products' unit
    unit = __builtin_ldexpf(a.scale * kLog2e, 20 + e - 11);
    half8_t t[KS];
    f.operands(e, t);
#pragma unroll
    for (int b = 0; b < G; ++b)
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        u32x4_t w = __builtin_bit_cast(u32x4_t, t[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = copy == b ? w[j] : 0u;
        q[b][i] = __builtin_bit_cast(half8_t, w);
      }
  }

  Acc<D> acc;
  acc.clear();
  if (any) {
    next = chunk(min(c_begin + kAttnWaves, c_end - 1), pg);
    auto step = [&](int ch, auto edge) {
      pages(min(ch + 2 * kAttnWaves, c_end - 1), pg);
      f32x4_t c[2][NG];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < NG; ++i) c[t][i] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < G; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < NG; ++i) {
              const u32x2_t w = k[b].pair(t, i);
              c[t][i] = mfma(e ? k_operand<true>(w.x, w.y) : k_operand<false>(w.x, w.y), q[b][2 * i + e], c[t][i]);
            }
#pragma unroll
      for (int b = 0; b < G; ++b) load_k<D>(next.at[b], lane, k[b]);
      const int t0 = (ch * G + copy) * kKv4Block + 4 * g;
      half8_t pf[kParts][NG];
      if constexpr (edge.value) {
        const Params<D> seen = drop_tail<D>(pr, t0, now.mine_there ? sr.len : 0);
        softmax_step<D, true, kTwo>(acc, c, RawParams<D>{seen, unit}, sumq, t0, now.mine_there ? lim : 0, pf);
      } else {
        softmax_step<D, false, kTwo>(acc, c, RawParams<D>{pr, unit}, sumq, t0, lim, pf);
      }
      load_p<D>(next.mine, g, pr);
#pragma unroll
      for (int b = 0; b < G; ++b)
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          half8_t pb[kParts];
#pragma unroll
          for (int h = 0; h < kParts; ++h) {
            u32x4_t pw = __builtin_bit_cast(u32x4_t, pf[h][i]);
            if constexpr (G > 1) {
#pragma unroll
              for (int j = 0; j < 4; ++j) pw[j] = copy == b ? pw[j] : 0u;
            }
            pb[h] = __builtin_bit_cast(half8_t, pw);
          }
#pragma unroll
          for (int j = 2 * i; j < 2 * i + 2; ++j) {
            const u32x2_t w = v[b].pair(j);
            const half8_t lo = v_operand<false>(w.x, w.y), hi = v_operand<true>(w.x, w.y);
#pragma unroll
            for (int h = 0; h < kParts; ++h) {
              acc.o[2 * j] = mfma(lo, pb[h], acc.o[2 * j]);
              acc.o[2 * j + 1] = mfma(hi, pb[h], acc.o[2 * j + 1]);
            }
          }
        }
#pragma unroll
      for (int b = 0; b < G; ++b) load_v<D>(next.at[b], lane, v[b]);
      now = next;
      next = chunk(min(ch + 2 * kAttnWaves, c_end - 1), pg);
    };
    const int whole = lim_lo / (G * kKv4Block);  // chunks that every row sees all of
    int ch = c_begin;
    for (; ch < min(whole, c_end) && now.all_there; ch += kAttnWaves) step(ch, std::false_type{});
    for (; ch < c_end; ch += kAttnWaves) step(ch, std::true_type{});
  }

  // join the waves and copies: every row's shares on a common maximum
  acc.finish();
  if (col % kRows < nrow) {
    if (g == 0) lds_m[wave][col] = acc.m, lds_l[wave][col] = acc.l;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f32x4_t t;
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = acc.value(i, j);
      *reinterpret_cast<f32x4_t*>(&lds_o[wave][col][16 * i + 4 * g]) = t;
    }
  }
  __syncthreads();
  for (int u = threadIdx.x; u < nrow * (D / 4); u += kAttnThreads) {
    const int r = u / (D / 4), d = 4 * (u % (D / 4));
    float m = kNoMax, l = 0.0f, o[4] = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kAttnWaves * G; ++w) m = fmaxf(m, lds_m[w / G][r + kRows * (w % G)]);
#pragma unroll
    for (int w = 0; w < kAttnWaves * G; ++w) {
      const int cc = r + kRows * (w % G);
      const float f = __builtin_amdgcn_exp2f(lds_m[w / G][cc] - m);
      l = __builtin_fmaf(f, lds_l[w / G][cc], l);
      const f32x4_t t = *reinterpret_cast<const f32x4_t*>(&lds_o[w / G][cc][d]);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __builtin_fmaf(f, t[j], o[j]);
    }
    const int rr = row0 + r, ti = a.by_group(rr);
    store_row<D, DT>(a, split, sr.first + ti, kvh * a.group + (rr - ti * a.group), d, o, m, l);
  }
}

// ---- more rows: a wave takes R tiles of 16 rows of its own ----
//
// Here the products and the softmax are the work, so a block is unpacked once
// for the workgroup's 64 R rows: each wave makes a quarter of the K and V
// operands and of the parameters (fp32, the score scale in K's scale), in LDS in the
// order of the product's lanes (16-byte accesses without conflicts).  Two
// buffers: while block b is used, block b + 1 is unpacked behind it and the
// codes of b + 2 are loaded; one barrier a block.
//
// Bound by the vector unit: the softmax is 7 operations and an exponential a
// score, 87 instructions a lane beside 8 matrix products for a tile of 16 rows x
// 32 tokens at D = 64 (vector unit 67 % busy, matrix unit 23 %).  2048 tokens of
// 32 heads over 8192, D = 64: 219 us with its join (14 us, two splits), 550
// Tflop/s; five ragged prompts, D = 128, bf16: 113 us, 510.
template <int D>
struct RowsBuf {
  u32x4_t k[2 * D / 32][kWave], v[D / 16][kWave];
  float par[4 * (D / 64)][kKv4Block];  // [group, kind][lane group's eight tokens in turn]
};

template <int D, int DT, int R>
__global__ __launch_bounds__(kAttnThreads, 2) void kv4_attn_rows_kernel(AttnArgs a) {
  using L = Kv4Layout<D>;
  constexpr int NG = D / 64, KS = D / 32, NT = D / 16;
  constexpr int kRows = 16 * R * kAttnWaves;
  __shared__ RowsBuf<D> lds[2];
  // the queries of two tiles at D = 128 would not fit the registers of two waves
  constexpr bool kLdsQ = D == 128 && R > 1;
  __shared__ u32x4_t lds_q[kLdsQ ? kAttnWaves : 1][kLdsQ ? R : 1][kLdsQ ? KS : 1][kWave];
  const Place at_place = place(a);
  const int split = at_place.split, seq = at_place.seq, kvh = at_place.head;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & (kWave - 1);
  const int col = lane & 15, g = lane >> 4;
  const SeqRange sr = seq_range(a, seq);
  const int rows = min(sr.n, a.max_q) * a.group;
  const int wg0 = at_place.tile * kRows;
  if (wg0 >= rows) return;
  const int row0 = wg0 + wave * 16 * R;
  const bool has_rows = row0 < rows;  // a wave without rows still unpacks
  auto limit = [&](int row) { return max(min(sr.len - sr.n + a.by_group(row) + 1, sr.len), 0); };
  const int lim_lo = limit(wg0), lim_hi = limit(min(wg0 + kRows, rows) - 1);
  const int wave_hi = limit(min(row0 + 16 * R, rows) - 1);

  const int nblk = (lim_hi + kKv4Block - 1) / kKv4Block;
  const int per = (nblk + a.splits - 1) / a.splits;
  const int b_begin = split * per, b_end = min(nblk, b_begin + per);
  const int page_blocks = a.c.page_shift - 5;
  const SHERRY_GLOBAL int32_t* table = gmem(a.table) + static_cast<int64_t>(seq) * a.table_stride;
  auto block = [&](int at, bool& there) {  // one that is not there reads the cache's first
    const int b = min(at, b_end - 1);      // (past the last: the last again)
    const int32_t pg = table[b >> page_blocks];
    there = pg >= 0 && pg < a.c.n_pages;
    const int64_t off = kv4_block_off<D>(a.c, there ? pg : 0, kvh, b & ((1 << page_blocks) - 1));
    return gmem(static_cast<const uint8_t*>(a.c.data)) + (there ? off : 0);
  };
  // the wave's share of a block: a pair of dwords a lane of K and of V (at
  // D = 64 of one of them), and of the parameters one value a thread
  constexpr bool kBoth = D == 128;
  const int share = kBoth ? wave : wave & 1;
  const bool does_k = kBoth || wave < 2, does_v = kBoth || wave >= 2;
  const int k_at = D == 64 ? lane * 16 + share * 8 : (share >> 1) * 1024 + lane * 16 + (share & 1) * 8;
  const int v_at = L::kVOff + (share >> 1) * 1024 + lane * 16 + (share & 1) * 8;
  const int kind = (threadIdx.x >> 5) & 3, idx = threadIdx.x & 31;
  const bool does_p = threadIdx.x < NG * 128;
  const int p_at = L::kPOff + (threadIdx.x >> 7) * 256 + idx * 2;
  u32x2_t kw = {0, 0}, vw = {0, 0};
  uint16_t p0 = 0, p1 = 0;
  auto fetch = [&](const SHERRY_GLOBAL uint8_t* blk) {
    if (does_k) kw = *reinterpret_cast<const SHERRY_GLOBAL u32x2_t*>(blk + k_at);
    if (does_v) vw = *reinterpret_cast<const SHERRY_GLOBAL u32x2_t*>(blk + v_at);
    if (does_p) {
      p0 = *reinterpret_cast<const SHERRY_GLOBAL uint16_t*>(blk + p_at + kind * 64);
      p1 = *reinterpret_cast<const SHERRY_GLOBAL uint16_t*>(blk + p_at + (kind >> 1) * 128);  // its scale
    }
  };
  const float unit = a.scale * kLog2e;
  auto unpack = [&](int b, RowsBuf<D>& to) {
    if (does_k) {
      // products of K: half block t, group gr -> operands 2 gr (low nibbles) and 2 gr + 1
      const int t = D == 64 ? share : share >> 1, gr = D == 64 ? 0 : share & 1;
      to.k[t * KS + 2 * gr][lane] = k_plus_base<DT, false>(kw.x, kw.y);
      to.k[t * KS + 2 * gr + 1][lane] = k_plus_base<DT, true>(kw.x, kw.y);
    }
    if (does_v) {
      to.v[2 * share][lane] = __builtin_bit_cast(u32x4_t, v_operand<false>(vw.x, vw.y));
      to.v[2 * share + 1][lane] = __builtin_bit_cast(u32x4_t, v_operand<true>(vw.x, vw.y));
    }
    if (does_p) {
      // tokens past the sequence may hold anything: their parameters are 0
      const int tok = b * kKv4Block + 16 * ((idx >> 2) & 1) + 4 * (idx >> 3) + (idx & 3);
      const float x = static_cast<float>(__builtin_bit_cast(_Float16, p0));
      const float s = static_cast<float>(__builtin_bit_cast(_Float16, p1));
      const float v = kind & 1 ? __builtin_fmaf(s, kind == 1 ? -kBase : kMid, x) : (kind == 0 ? x * unit : x);
      to.par[(threadIdx.x >> 7) * 4 + kind][idx] = tok < sr.len ? v : 0.0f;
    }
  };
  bool now_there = false, next_there = false;
  if (b_begin < b_end) fetch(block(b_begin, now_there));

  u32x4_t q[R][KS];
  float sumq[R][NG];
  int lim[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = min(row0 + 16 * r + col, rows - 1);
    const int tok = a.by_group(row), head = kvh * a.group + (row - tok * a.group);
    lim[r] = sr.len - sr.n + tok + 1;
    Queries<D, DT> f;
    f.load(a.q, (sr.first + tok) * a.q_st + head * a.q_sh + 8 * g);
    f.sums(unit, sumq[r]);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      q[r][i] = f.bits(i);
      if constexpr (kLdsQ) lds_q[wave][r][i][lane] = q[r][i];  // (read by the wave that writes them)
    }
  }
  Acc<D> acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r].clear();
  if (b_begin < b_end) {
    unpack(b_begin, lds[0]);
    fetch(block(b_begin + 1, next_there));
    __syncthreads();
  }

  auto step = [&](int b, auto edge) {
    const int turn = b - b_begin;
    const RowsBuf<D>& from = lds[turn & 1];
    if (now_there && has_rows && (!edge.value || b * kKv4Block < wave_hi)) {
      f32x4_t c[R][2][NG];
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          u32x4_t qi[R];
#pragma unroll
          for (int r = 0; r < R; ++r) qi[r] = kLdsQ ? lds_q[wave][r][2 * i + e][lane] : q[r][2 * i + e];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const u32x4_t k = from.k[t * KS + 2 * i + e][lane];
#pragma unroll
            for (int r = 0; r < R; ++r) c[r][t][i] = mfma_k<DT>(k, qi[r], e ? c[r][t][i] : f32x4_t{0, 0, 0, 0});
          }
        }
      const int t0 = b * kKv4Block + 4 * g;
      half8_t pf[R][1][NG];
#pragma unroll
      for (int r = 0; r < R; ++r)
        softmax_step<D, edge.value, false>(acc[r], c[r], LdsParams<D>{&from.par[0][8 * g]}, sumq[r], t0, lim[r], pf[r]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const half8_t v = __builtin_bit_cast(half8_t, from.v[i][lane]);
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r].o[i] = mfma(v, pf[r][0][i >> 2], acc[r].o[i]);
      }
    }
    now_there = next_there;
    if (b + 1 < b_end) {
      unpack(b + 1, lds[(turn + 1) & 1]);
      fetch(block(b + 2, next_there));
      __syncthreads();
    }
  };
  const int whole = lim_lo / kKv4Block;  // blocks that every row sees all of
  int b = b_begin;
  for (; b < min(whole, b_end); ++b) step(b, std::false_type{});
  for (; b < b_end; ++b) step(b, std::true_type{});
#pragma unroll
  for (int r = 0; r < R; ++r) {
    acc[r].finish();
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = acc[r].value(i, j);
    const int row = row0 + 16 * r + col;
    if (row >= rows) continue;
    const int tok = a.by_group(row), head = kvh * a.group + (row - tok * a.group);
#pragma unroll
    for (int i = 0; i < NT; ++i) store_row<D, DT>(a, split, sr.first + tok, head, 16 * i + 4 * g, o[i], acc[r].m, acc[r].l);
  }
}

// Joins the splits of every row.  A row takes D / 4 lanes (four values each)
// times 1 << sg_shift groups, and group i the splits i, i + groups, ..., four at a
// time, so that one latency covers up to 64 (D = 64) or 32 of them.
template <int D, int DT>
__global__ __launch_bounds__(kAttnThreads) void kv4_join_kernel(AttnArgs a, int join_blocks, int sg_shift) {
  constexpr int kLanes = D / 4;
  __shared__ f32x4_t lds_o[kAttnThreads];
  __shared__ f32x2_t lds_ml[kAttnThreads];
  const int seq = static_cast<int>(blockIdx.x / join_blocks);
  const SeqRange sr = new_range(a, seq);
  const int groups = 1 << sg_shift;
  const int lane = threadIdx.x % kLanes;
  const int grp = (threadIdx.x / kLanes) & (groups - 1);
  const int64_t u =
      (static_cast<int64_t>(blockIdx.x % join_blocks) * (kAttnThreads / kLanes) >> sg_shift) +
      (threadIdx.x / kLanes >> sg_shift);
  const int64_t ti = u / a.n_q_heads;
  const bool live = ti < min(sr.n, a.max_q);
  const int hd = static_cast<int>(u - ti * a.n_q_heads);
  const int64_t token = sr.first + ti;
  const int64_t at = token * a.n_q_heads + hd, step = a.n_tokens * a.n_q_heads;
  float m = kNoMax, l = 0.0f;
  f32x4_t v = {0, 0, 0, 0};
  if (live) {
    const SHERRY_GLOBAL f32x2_t* ml = gmem(reinterpret_cast<const f32x2_t*>(a.part_ml)) + at;
    const SHERRY_GLOBAL f32x4_t* po = gmem(reinterpret_cast<const f32x4_t*>(a.part_o)) + at * kLanes + lane;
    for (int s0 = grp; s0 < a.splits; s0 += 4 * groups) {
      f32x2_t t[4];
      f32x4_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // (past the last: the first again, with no weight)
        const int s = s0 + i * groups < a.splits ? s0 + i * groups : s0;
        t[i] = ml[s * step];
        o[i] = po[s * step * kLanes];
      }
      const float m_old = m;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, t[i].x);
      const float keep = __builtin_amdgcn_exp2f(m_old - m);
      l *= keep;
      v *= keep;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = s0 + i * groups < a.splits ? __builtin_amdgcn_exp2f(t[i].x - m) : 0.0f;
        l = __builtin_fmaf(f, t[i].y, l);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(f, o[i][j], v[j]);
      }
    }
  }
  if (groups > 1) {
    lds_o[threadIdx.x] = v;
    lds_ml[threadIdx.x] = f32x2_t{m, l};
    __syncthreads();
    if (grp != 0) return;
    for (int i = 1; i < groups; ++i) m = fmaxf(m, lds_ml[threadIdx.x + i * kLanes].x);
    l = 0.0f;
    v = f32x4_t{0, 0, 0, 0};
    for (int i = 0; i < groups; ++i) {
      const f32x2_t t = lds_ml[threadIdx.x + i * kLanes];
      const f32x4_t o = lds_o[threadIdx.x + i * kLanes];
      const float f = __builtin_amdgcn_exp2f(t.x - m);
      l = __builtin_fmaf(f, t.y, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(f, o[j], v[j]);
    }
  }
  if (!live) return;
  AttnArgs one = a;
  one.splits = 1;  // the final store
  const float o[4] = {v[0], v[1], v[2], v[3]};
  store_row<D, DT>(one, 0, token, hd, 4 * lane, o, m, l);
}

template <int D, int DT>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.splits) * a.n_seqs * a.row_tiles * a.c.n_kv_heads));
  const dim3 block(kAttnThreads);
  if (a.tile_rows == 8) hipLaunchKernelGGL((kv4_attn_few_kernel<D, DT, 2>), grid, block, 0, stream, a);
  else if (a.tile_rows == 16) hipLaunchKernelGGL((kv4_attn_few_kernel<D, DT, 1>), grid, block, 0, stream, a);
  else if (a.tile_rows == 16 * kAttnWaves) hipLaunchKernelGGL((kv4_attn_rows_kernel<D, DT, 1>), grid, block, 0, stream, a);
  else if (a.tile_rows == 32 * kAttnWaves) hipLaunchKernelGGL((kv4_attn_rows_kernel<D, DT, 2>), grid, block, 0, stream, a);
  else if constexpr (D == 64) hipLaunchKernelGGL((kv4_attn_rows_kernel<D, DT, 4>), grid, block, 0, stream, a);
  if (a.splits > 1) {
    int sg = 0;
    while (sg < (D == 64 ? 4 : 3) && (2 << sg) <= a.splits) ++sg;
    const int rows_per = kAttnThreads / (D / 4) >> sg;
    const int64_t jb = (static_cast<int64_t>(a.max_q) * a.n_q_heads + rows_per - 1) / rows_per;
    hipLaunchKernelGGL((kv4_join_kernel<D, DT>), dim3(static_cast<unsigned>(jb * a.n_seqs)), block, 0, stream, a,
                       static_cast<int>(jb), sg);
  }
  return hipGetLastError();
}

}  // namespace

// Rows per workgroup.  Up to 8 or 16 rows go to the kernel that shares out the
// cached tokens.  Beyond, 1, 2 or 4 tiles of 16 rows a wave (2 at most at D =
// 128, whose registers hold no more): a block's unpacking serves them all, but
// fewer, longer workgroups fill the chip less evenly, the more so where a
// prompt's first rows see little.  So one tile for short sequences (mean tokens
// seen below 1664) while the chip is filled no more than a few times over, and
// whenever one tile a wave does not fill half of it; four for long ones.  8 key
// heads, 4 query heads each, us with 1 / 2 / 4 tiles, prompts of q tokens (the
// last of ctx):
//   D = 64, q of ctx: 128 of 128  7 / 9 / 12      D = 128: 128 of 128  9 / 12
//     512 of 512     19 / 21 / 22                   512 of 512     23 / 27
//     2048 of 2048   51 / 61 / 67                   1024 of 2048   67 / 70
//     512 of 2048    36 / 32 / 45                   2048 of 4096   214 / 186
//     4096 of 4096   149 / 121 / 169                4096 of 4096   248 / 247
//     128 of 4096    27 / 30 / 33                   128 of 4096    39 / 39
//     2048 of 8192   254 / 253 / 219                512 of 8192    156 / 130
int32_t kv4_attn_tile_rows(int64_t rows, int64_t heads, int head_dim, int64_t max_q, int64_t max_kv) {
  if (rows <= 16) return rows <= 8 ? 8 : 16;
  constexpr int32_t one = 16 * kAttnWaves;
  const int64_t tiles = (rows + one - 1) / one * heads;
  const int64_t seen = std::max(max_kv - max_q / 2, max_q / 2);
  if (rows <= one || tiles <= 128 || (seen < 1664 && tiles * head_dim < 1536 * 64)) return one;
  if (head_dim == 128 || rows <= 2 * one || seen < 3328 || tiles < 512) return 2 * one;
  return 4 * one;
}

// Splits of the cached tokens.  The join costs about 4 us, so nothing is split
// that a workgroup does in that: 4 steps of its waves (few rows) or 8 blocks.
// Beyond, one workgroup a CU, down to one step or two blocks each; and where that
// leaves each enough, for uneven lengths and latency, two a CU (4 steps or 8
// blocks each) or 1536 workgroups (8 steps), but no number between, which would
// fill some CUs only (40000 tokens: 13.6 us with 40 splits).
// Measured, us, 8 key heads, with 1 / 2 / 4 ... splits:
//   one token, D = 64, over 1000: 7.5 / 8.5 / 8.0 / 8.4
//     over 4000: 17.6 / 13.5 / 10.6 / 9.4 / 8.7 / 8.6 / 8.8 (64)
//     over 40000: 133 / 72 / 40 / 24 / 16.4 / 12.4 / 12.7
//     over 131072: 23.5 / 22.0 / 21.7 with 32 / 64 / 128
//   9 of 5 tokens over up to 4099, 16 key heads, D = 128: 20.9 / 21.5 / 19.5 /
//     20.5 / 22.5 with 2 / 3 / 4 / 5 / 6
//   48 uneven ones, D = 128: 92 / 86 / 82 / 82 / 85 with 2 / 3 / 4 / 5 / 6
//   20 rows, D = 64, over 1000: 24.7 / 17.1 / 12.2 / 10.2 / 9.0 / 8.7 (32)
//   64 rows, D = 128, over 4000: 115 / 63 / 37 / 24 / 17.3 / 16.4 / 20.9 (64)
//   8192 rows over 8192 (256 workgroups): 322 / 219 / 224 (4)
// The workspace of any call is bounded by that: with 512 workgroups aimed at, a
// split call of n < 512 has fewer than 512 + n <= 1023 of them, of up to 256 rows
// of 64 + 2 floats or 128 of 128 + 2; of few rows fewer than 3072, of 16.
static_assert(1023 * 256 * (64 + 2) * 4 <= SHERRY_KV4_ATTN_WORKSPACE_MAX &&
              1023 * 128 * (128 + 2) * 4 <= SHERRY_KV4_ATTN_WORKSPACE_MAX &&
              3071 * 16 * (128 + 2) * 4 <= SHERRY_KV4_ATTN_WORKSPACE_MAX);
int32_t kv4_attn_splits(int32_t tile_rows, int64_t workgroups, int64_t max_kv) {
  const bool few = tile_rows <= 16;
  const int64_t step = few ? int64_t(kAttnWaves) * (16 / tile_rows) * kKv4Block : kKv4Block;
  if (max_kv <= (few ? 4 : 8) * step) return 1;
  auto splits_to = [&](int64_t total) { return (total + workgroups - 1) / workgroups; };
  const int64_t least = few ? step : 2 * step;
  int64_t n = std::min(splits_to(256), (max_kv + least - 1) / least);
  const int64_t two = splits_to(512), six = splits_to(1536);
  if (max_kv >= two * (few ? 4 : 8) * step) n = two;
  if (few && max_kv >= six * 8 * step) n = six;
  return static_cast<int32_t>(n);
}

hipError_t launch_kv4_attn(const AttnArgs& a, int head_dim, int dt, hipStream_t stream) {
  if (head_dim == 64) return dt == kActF16 ? launch_d<64, kActF16>(a, stream) : launch_d<64, kActBf16>(a, stream);
  return dt == kActF16 ? launch_d<128, kActF16>(a, stream) : launch_d<128, kActBf16>(a, stream);
}

}  // namespace sherry
