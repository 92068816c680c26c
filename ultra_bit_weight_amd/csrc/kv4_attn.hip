// Attention of new tokens over the 4-bit key/value cache.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j,  j <= position of i
//
// and, with a window, only j > position - window or j < sinks: the blocks between
// the sinks and the first row's window are not walked (see Walk).
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

// The blocks of cached tokens that a workgroup walks, numbered without a gap.
// With a window these are the blocks that hold sinks, then those from the first
// row's window on; without one, all of them up to the last row's position.
// `whole` to `whole_end`: blocks of which every row sees all, from the last row's window
// on.  (Blocks of sinks before it are tested score by score, those too of which every row
// sees all: 2048 tokens over 8192, D = 64, 40.4 us with a window of 1000 and 20 sinks, 48.6
// with 200, where a window of 1200 takes 44.2, and 81 with 1000, one of 2000 66.)
template <bool kWin>
struct Walk {
  int n;                 // blocks
  int whole, whole_end;
  int head, gap;         // blocks before the gap, and blocks left out
  int low, sinks;        // no row sees tokens sinks .. low - 1
  // lim_lo, lim_hi: how many tokens there are up to the first and the last row's own
  __device__ __forceinline__ Walk(const AttnArgs& a, int lim_lo, int lim_hi) {
    n = (lim_hi + kKv4Block - 1) / kKv4Block;
    whole = 0, whole_end = lim_lo / kKv4Block;
    head = gap = low = sinks = 0;
    if constexpr (kWin) {
      sinks = a.sinks;
      low = max(lim_lo - a.window, 0);
      head = (min(sinks, lim_hi) + kKv4Block - 1) / kKv4Block;
      gap = max(low / kKv4Block - head, 0);
      const int low_last = max(lim_hi - a.window, 0);  // where the last row's window begins
      whole = low_last <= sinks ? 0 : (low_last + kKv4Block - 1) / kKv4Block - gap;
      n -= gap;
      whole_end -= gap;
    }
  }
  __device__ __forceinline__ int block(int b) const {  // its number in the sequence
    if constexpr (kWin) return b < head ? b : b + gap;
    return b;
  }
  __device__ __forceinline__ bool seen(int t, int len) const {  // by any row, as far as its place in the walk says
    if constexpr (kWin) return t < len && (t >= low || t < sinks);
    return t < len;
  }
};

// Zeroes the scales of tokens that no row sees (their bytes may be anything, and
// 0 * NaN is not 0): those past `len`, and with a window those before it that are
// no sinks; t0 is the lane's first token.
template <int D, bool kWin>
__device__ __forceinline__ Params<D> drop_unseen(Params<D> p, const Walk<kWin>& walk, int t0, int len) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + 16 * (i >> 1) + 2 * (i & 1);
    const uint32_t mask = (walk.seen(t, len) ? 0xFFFFu : 0u) | (walk.seen(t + 1, len) ? 0xFFFF0000u : 0u);
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

// What a row sees: tokens below lim, with a window only from low on or below sinks.
template <bool kWin>
struct Sees {
  int lim, low, sinks;
  __device__ __forceinline__ bool operator()(int t) const {
    if constexpr (kWin) return t < lim && (t >= low || t < sinks);
    return t < lim;
  }
};
template <bool kWin>
__device__ __forceinline__ Sees<kWin> sees_of(const AttnArgs& a, int lim) {
  return {lim, max(lim, 0) - a.window, a.sinks};  // (not used without a window)
}

// The softmax step of one tile: scores from the products c (S^T of each scale
// group) to P operands, one per group.  kEdge: not every token is seen (t0 is the
// lane's first one).
template <int D, bool kEdge, bool kTwo, bool kWin, class P>
__device__ __forceinline__ void softmax_step(Acc<D>& a, const f32x4_t (&c)[2][D / 64], const P& pr,
                                             const float (&sumq)[D / 64], int t0, const Sees<kWin>& sees,
                                             half8_t (&pf)[kTwo ? 2 : 1][D / 64]) {
  constexpr int NG = D / 64;
  constexpr bool kReady = std::is_same_v<P, LdsParams<D>>;  // the unit is in the parameters
  float p[8], ps[NG][8], top, sum;
  // The maximum is taken off the rounded score that it was taken of.  Folded into
  // the first fma it would round apart from that, by units from scores (or parts
  // of scores) of 2^24 on, and the largest weight be infinite or 0; the operation
  // costs 219 us against 213 for 2048 tokens over 8192, 113.1 against 112.0 for
  // ragged prompts, and where rows are few 1 % at most (12.2 against 12.0 for one
  // token over 40000; 21.2 and 82.8 for 131072 and a batch as before).  Folded only
  // where the maximum stays, nothing is infinite, but from scores of about 2^20 on
  // equal keys weigh apart by where they lie (2048 tokens over 8192, D = 64, windows of
  // 1000, 2048 and 4096 43.1, 65.2 and 117 us, 44.1, 67.4 and 122 as here).
  auto score = [&](int i, float m) {
    float u = pr.kz(0, i) * sumq[0];
#pragma unroll
    for (int k = 1; k < NG; ++k) u = __builtin_fmaf(pr.kz(k, i), sumq[k], u);
#pragma unroll
    for (int k = 0; k < NG; ++k) u = __builtin_fmaf(pr.ks(k, i), c[i >> 2][k][i & 3], u);
    if constexpr (!kReady) u *= pr.unit;
    u -= m;
    if constexpr (kEdge) u = sees(t0 + 16 * (i >> 2) + (i & 3)) ? u : -__builtin_inff();
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
template <int D, int DT, int G, bool kWin>
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

  const Walk<kWin> walk(a, max(sr.len - sr.n + a.by_group(row0) + 1, 0),
                        max(min(sr.len - sr.n + a.by_group(row0 + nrow - 1) + 1, sr.len), 0));
  const int row = min(row0 + col % kRows, rows - 1);
  const int tok = a.by_group(row);
  const int head = kvh * a.group + (row - tok * a.group);
  const Sees<kWin> sees = sees_of<kWin>(a, sr.len - sr.n + tok + 1);

  const int nblk = walk.n;
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
    for (int b = 0; b < G; ++b) pg[b] = table[walk.block(min(ch * G + b, nblk - 1)) >> page_blocks];
  };
  auto chunk = [&](int ch, const int32_t (&pg)[G]) {
    Chunk c;
    c.all_there = true;
#pragma unroll
    for (int b = 0; b < G; ++b) {
      const int blk = walk.block(ch * G + b);
      const bool there = ch * G + b < nblk && pg[b] >= 0 && pg[b] < a.c.n_pages;
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
      const int t0 = walk.block(ch * G + copy) * kKv4Block + 4 * g;
      half8_t pf[kParts][NG];
      if constexpr (edge.value) {
        const Params<D> seen = drop_unseen<D, kWin>(pr, walk, t0, now.mine_there ? sr.len : 0);
        softmax_step<D, true, kTwo, kWin>(acc, c, RawParams<D>{seen, unit}, sumq, t0,
                                          Sees<kWin>{now.mine_there ? sees.lim : 0, sees.low, sees.sinks}, pf);
      } else {
        softmax_step<D, false, kTwo, kWin>(acc, c, RawParams<D>{pr, unit}, sumq, t0, sees, pf);
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
    const int whole = (walk.whole + G - 1) / G, whole_end = walk.whole_end / G;  // chunks that every row sees all of
    int ch = c_begin;
    if constexpr (kWin)
      for (; ch < min(whole, c_end); ch += kAttnWaves) step(ch, std::true_type{});
    for (; ch < min(whole_end, c_end) && now.all_there; ch += kAttnWaves) step(ch, std::false_type{});
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
        softmax_step<D, edge.value, false, false>(acc[r], c[r], LdsParams<D>{&from.par[0][8 * g]}, sumq[r], t0,
                                                  Sees<false>{lim[r], 0, 0}, pf[r]);
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

// ---- more rows with a window ----
//
// The same step, for W waves of one tile each.  A row sees about as much as any
// other, so workgroups are alike and there are many: what counts is how few
// instructions a row takes, and that enough waves are there to fill each other's
// waits.  Eight waves (D = 64) halve the unpacking of each, and its page numbers,
// branches and barriers: a step is two blocks, one unpacked by each half of the
// waves.  Two or four tiles a wave share the unpacking too, but leave two waves to a
// vector unit instead of four.  Bound by a wave's chain of unpacking, products and
// softmax, which four waves a vector unit (D = 128: three) do not hide whole, and by
// the blocks at either end of a tile's window, whose scores are tested one by one:
// neither unit is full (vector 59 %, matrix 15 % busy of a 2048-token chunk, window 1000),
// and a wave waits for 39 % of its cycles.
// P enters the second product as one fp16 operand (2^-11 of each weight), as without a
// window: of fp16 results the error is 3.0e-4 against 2.1e-4 of the result's own rounding,
// which a second operand for P's rounding error comes down to, at 50.9 us against 44.7
// (window 1000, 20 sinks), 99 against 91 (five prompts, D = 128); of bf16 results 1.66e-3
// against 1.64e-3.
// 2048 tokens of 32 heads on 8 over 8192, D = 64, us, with one / two / four tiles
// on four waves, and with eight waves: window 1000 48.1 / 47.7 / 63.0, 42.9; 4096
// 158 / 155 / 144, 137; and with the softmax's wave priority 41.9 and 130, with page
// numbers of 64 blocks at once 39.9 and 123 (570 Tflop/s); sixteen waves no faster.
// D = 128, five prompts of up to 1777 with a window of 512: 87.2 / 94.2; eight waves
// 95.6, their registers spilled; with page numbers of 64 blocks 85.3; with the priority
// 1 % more, but 2048 tokens over 8192, windows of 512, 1000 and 4096, 37.6, 58.4, 196
// -> 35.7, 55.7, 185.
template <int D, int DT, int W>
__global__ __launch_bounds__(W * kWave, W == 8 ? 4 : D == 128 ? 3 : 2) void kv4_attn_window_rows_kernel(AttnArgs a) {
  using L = Kv4Layout<D>;
  static_assert(W == kAttnWaves || (W == 2 * kAttnWaves && D == 64));
  constexpr int NG = D / 64, KS = D / 32, NT = D / 16;
  constexpr int kRows = 16 * W, kPer = W / kAttnWaves;  // blocks of a step
  __shared__ RowsBuf<D> lds[2][kPer];
  const Place at_place = place(a);
  const int split = at_place.split, seq = at_place.seq, kvh = at_place.head;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & (kWave - 1);
  const int col = lane & 15, g = lane >> 4;
  const SeqRange sr = seq_range(a, seq);
  const int rows = min(sr.n, a.max_q) * a.group;
  const int wg0 = at_place.tile * kRows;
  if (wg0 >= rows) return;
  const int row0 = wg0 + wave * 16;
  const bool has_rows = row0 < rows;  // a wave without rows still unpacks
  auto limit = [&](int row) { return max(min(sr.len - sr.n + a.by_group(row) + 1, sr.len), 0); };
  const Walk<true> walk(a, limit(wg0), limit(min(wg0 + kRows, rows) - 1));
  // the wave's rows see no token from hi on, nor those between the sinks and low
  const int hi = limit(min(row0 + 16, rows) - 1), low = limit(min(row0, rows - 1)) - a.window;

  const int per = (walk.n + a.splits - 1) / a.splits;
  const int b_begin = split * per, b_end = min(walk.n, b_begin + per);
  const int page_blocks = a.c.page_shift - 5;
  const SHERRY_GLOBAL int32_t* table = gmem(a.table) + static_cast<int64_t>(seq) * a.table_stride;
  // Page numbers, a block a lane, of 64 blocks from `held` on; -1 for one that is no
  // page.  (Past the last block: the last again; a block that is not there reads the
  // cache's first.)  A load of each step's own, being one number for the wave, is
  // waited for where it stands and the codes' loads with it: 41.9 against 39.9 us for
  // 2048 tokens and a window of 1000, 129.6 against 122.7 for 4096 (D = 64), 200.4
  // against 195.8 (D = 128).
  int held = 0;
  int32_t page_of = -1;
  auto hold = [&](int b) {
    held = b;
    const int32_t pg = table[walk.block(min(b + lane, b_end - 1)) >> page_blocks];
    page_of = pg >= 0 && pg < a.c.n_pages ? pg : -1;
  };
  auto pages = [&](int b, int32_t (&pg)[kPer]) {
    if (b + kPer > held + kWave) hold(b);
#pragma unroll
    for (int i = 0; i < kPer; ++i) pg[i] = __builtin_amdgcn_readlane(page_of, b + i - held);
  };
  // the wave's share: of block `sub` of a step, a pair of dwords a lane of K and of V
  // (D = 64: of one of them), and of the parameters one value a thread
  constexpr bool kBoth = D == 128;
  const int sub = wave / kAttnWaves, part = wave & (kAttnWaves - 1);
  const int share = kBoth ? part : part & 1;
  const bool does_k = kBoth || part < 2, does_v = kBoth || part >= 2;
  const int k_at = D == 64 ? lane * 16 + share * 8 : (share >> 1) * 1024 + lane * 16 + (share & 1) * 8;
  const int v_at = L::kVOff + (share >> 1) * 1024 + lane * 16 + (share & 1) * 8;
  const int thread = threadIdx.x & (kAttnThreads - 1);
  const int kind = (thread >> 5) & 3, idx = thread & 31, group = thread >> 7;
  const bool does_p = thread < NG * 128;
  const int p_at = L::kPOff + group * 256 + idx * 2;
  u32x2_t kw = {0, 0}, vw = {0, 0};
  uint16_t p0 = 0, p1 = 0;
  auto fetch = [&](int b, const int32_t (&pg)[kPer]) {
    const int32_t mine = kPer == 1 || sub == 0 ? pg[0] : pg[kPer - 1];
    const int in_page = walk.block(min(b + sub, b_end - 1)) & ((1 << page_blocks) - 1);
    const int64_t off = mine >= 0 ? kv4_block_off<D>(a.c, mine, kvh, in_page) : 0;
    const SHERRY_GLOBAL uint8_t* blk = gmem(static_cast<const uint8_t*>(a.c.data)) + off;
    if (does_k) kw = *reinterpret_cast<const SHERRY_GLOBAL u32x2_t*>(blk + k_at);
    if (does_v) vw = *reinterpret_cast<const SHERRY_GLOBAL u32x2_t*>(blk + v_at);
    if (does_p) {
      p0 = *reinterpret_cast<const SHERRY_GLOBAL uint16_t*>(blk + p_at + kind * 64);
      p1 = *reinterpret_cast<const SHERRY_GLOBAL uint16_t*>(blk + p_at + (kind >> 1) * 128);  // its scale
    }
  };
  const float unit = a.scale * kLog2e;
  auto unpack = [&](int b, RowsBuf<D> (&step)[kPer]) {
    RowsBuf<D>& to = step[kPer == 1 ? 0 : sub];
    if (does_k) {
      const int t = D == 64 ? share : share >> 1, gr = D == 64 ? 0 : share & 1;
      to.k[t * KS + 2 * gr][lane] = k_plus_base<DT, false>(kw.x, kw.y);
      to.k[t * KS + 2 * gr + 1][lane] = k_plus_base<DT, true>(kw.x, kw.y);
    }
    if (does_v) {
      to.v[2 * share][lane] = __builtin_bit_cast(u32x4_t, v_operand<false>(vw.x, vw.y));
      to.v[2 * share + 1][lane] = __builtin_bit_cast(u32x4_t, v_operand<true>(vw.x, vw.y));
    }
    if (does_p) {
      // tokens that no row sees may hold anything: their parameters are 0
      const int tok = walk.block(b + sub) * kKv4Block + 16 * ((idx >> 2) & 1) + 4 * (idx >> 3) + (idx & 3);
      const float x = static_cast<float>(__builtin_bit_cast(_Float16, p0));
      const float s = static_cast<float>(__builtin_bit_cast(_Float16, p1));
      const float v = kind & 1 ? __builtin_fmaf(s, kind == 1 ? -kBase : kMid, x) : (kind == 0 ? x * unit : x);
      to.par[group * 4 + kind][idx] = walk.seen(tok, sr.len) ? v : 0.0f;
    }
  };
  int32_t now[kPer], next[kPer];
  const bool any = b_begin < b_end;
  if (any) {
    hold(b_begin);
    pages(b_begin, now);
    fetch(b_begin, now);
  }

  u32x4_t q[KS];
  float sumq[NG];
  Sees<true> sees;
  {
    const int row = min(row0 + col, rows - 1);
    const int tok = a.by_group(row), head = kvh * a.group + (row - tok * a.group);
    sees = sees_of<true>(a, sr.len - sr.n + tok + 1);
    Queries<D, DT> f;
    f.load(a.q, (sr.first + tok) * a.q_st + head * a.q_sh + 8 * g);
    f.sums(unit, sumq);
#pragma unroll
    for (int i = 0; i < KS; ++i) q[i] = f.bits(i);
  }
  Acc<D> acc;
  acc.clear();
  if (any) {
    unpack(b_begin, lds[0]);
    pages(b_begin + kPer, next);
    fetch(b_begin + kPer, next);
    __syncthreads();
  }

  auto block_step = [&](const RowsBuf<D>& from, int t_blk, auto edge) {
    constexpr bool kFirst = !edge.value;
    f32x4_t c[2][NG];
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          c[t][i] = mfma_k<DT>(from.k[t * KS + 2 * i + e][lane], q[2 * i + e], e ? c[t][i] : f32x4_t{0, 0, 0, 0});
    half8_t pf[1][NG];
    // a wave that has its scores goes on to their product before others begin theirs
    if constexpr (kFirst) __builtin_amdgcn_s_setprio(1);
    softmax_step<D, edge.value, false, true>(acc, c, LdsParams<D>{&from.par[0][8 * g]}, sumq, t_blk + 4 * g, sees, pf);
#pragma unroll
    for (int i = 0; i < NT; ++i)
      acc.o[i] = mfma(__builtin_bit_cast(half8_t, from.v[i][lane]), pf[0][i >> 2], acc.o[i]);
    if constexpr (kFirst) __builtin_amdgcn_s_setprio(0);
  };
  auto step = [&](int b, int turn, auto edge) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t_blk = walk.block(b + i) * kKv4Block;
      if (has_rows && now[i] >= 0 &&
          (!edge.value || (b + i < b_end && t_blk < hi && (t_blk + kKv4Block > low || t_blk < a.sinks))))
        block_step(lds[turn & 1][i], t_blk, edge);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) now[i] = next[i];
    if (b + kPer < b_end) {
      unpack(b + kPer, lds[(turn + 1) & 1]);
      pages(b + 2 * kPer, next);
      fetch(b + 2 * kPer, next);
      __syncthreads();
    }
  };
  int b = b_begin, turn = 0;
  for (; b < min(walk.whole, b_end); b += kPer) step(b, turn++, std::true_type{});
  for (; b + kPer <= min(walk.whole_end, b_end); b += kPer) step(b, turn++, std::false_type{});
  for (; b < b_end; b += kPer) step(b, turn++, std::true_type{});

  acc.finish();
  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = acc.value(i, j);
  const int row = row0 + col;
  if (row >= rows) return;
  const int tok = a.by_group(row), head = kvh * a.group + (row - tok * a.group);
#pragma unroll
  for (int i = 0; i < NT; ++i) store_row<D, DT>(a, split, sr.first + tok, head, 16 * i + 4 * g, o[i], acc.m, acc.l);
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

template <int D, int DT, bool kWin>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.splits) * a.n_seqs * a.row_tiles * a.c.n_kv_heads));
  const dim3 block(kAttnThreads);
  if (a.tile_rows == 8) hipLaunchKernelGGL((kv4_attn_few_kernel<D, DT, 2, kWin>), grid, block, 0, stream, a);
  else if (a.tile_rows == 16) hipLaunchKernelGGL((kv4_attn_few_kernel<D, DT, 1, kWin>), grid, block, 0, stream, a);
  else if constexpr (kWin) {
    if (a.tile_rows == 16 * kAttnWaves)
      hipLaunchKernelGGL((kv4_attn_window_rows_kernel<D, DT, kAttnWaves>), grid, block, 0, stream, a);
    else if constexpr (D == 64)
      hipLaunchKernelGGL((kv4_attn_window_rows_kernel<D, DT, 2 * kAttnWaves>), grid, dim3(2 * kAttnThreads), 0, stream, a);
  }
  else if (a.tile_rows == 16 * kAttnWaves) hipLaunchKernelGGL((kv4_attn_rows_kernel<D, DT, 1>), grid, block, 0, stream, a);
  else if (a.tile_rows == 32 * kAttnWaves) hipLaunchKernelGGL((kv4_attn_rows_kernel<D, DT, 2>), grid, block, 0, stream, a);
  else if constexpr (D == 64) hipLaunchKernelGGL((kv4_attn_rows_kernel<D, DT, 4>), grid, block, 0, stream, a);
  if (a.splits > 1) {
    int sg = 0;
    while (sg < (D == 64 ? 4 : 3) && (2 << sg) <= a.splits) ++sg;
    // With a window groups of four splits each, since what those that are not there
    // load (the first again) counts where rows are many.  (Two groups at D = 64 are
    // slower than one or four: 37.2 against 32.2 us for 512 tokens in six splits.)
    if constexpr (kWin) {
      sg = 0;
      while (sg < (D == 64 ? 4 : 3) && 4 << sg < a.splits) ++sg;
      if (D == 64 && sg == 1) sg = 2;
    }
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

// With a window the kernel that shares out the tokens takes more rows too, 16 a
// workgroup, where those are so few, or see so little, that what counts is how soon
// each is through, not that every 16 rows unpack their tokens for themselves.  Beyond,
// eight waves a workgroup where the registers allow it (D = 64) and that leaves a
// workgroup a CU (512 tokens over 2048, window 256: 18.5 us with eight, 12.6 with four).
// us, shared out / by rows, workgroups of 16 rows in brackets, windows of 100, 500, 2000
// and 6000:
//   D = 64, 32 rows [16]     5.4 / 8.5, 6.9 / 9.1, 7.9 / 10.4, 9.1 / 12.9
//           32 rows [1024]   8.3 / 10.6, 13.4 / 18.2, 34.4 / 46.9, 86 / 123
//           64 rows [768]    7.4 / 8.9, 11.6 / 20.7, 26.1 / 30.6, 65 / 56
//           64 rows [2048]   13.8 / 11.0, 23.4 / 20.2, 62.9 / 48.2
//           256 rows [128]   5.8 / 9.6, 7.3 / 10.9, 11.9 / 13.6, 18.7 / 25.6
//           384 rows [192]   5.8 / 9.6, 7.4 / 11.4, 15.6 / 15.6, 27.0 / 22.7
//   D = 128, 48 rows [24]    7.0 / 10.1, 9.6 / 10.8, 11.7 / 13.2, 15.2 / 17.0
//           126 rows [384]   8.9 / 12.0, 13.7 / 19.7, 29.1 / 32.4, 72 / 52
//           63 rows [768]    13.1 / 10.8, 18.8 / 23.2, 44.6 / 41.5
int32_t kv4_attn_window_tile_rows(int64_t rows, int64_t heads, int head_dim, int64_t seen) {
  if (rows <= 16) return rows <= 8 ? 8 : 16;
  const int64_t few = (rows + 15) / 16 * heads;
  const bool wide = head_dim == 128;
  if ((rows <= 32 && !wide) || few <= (wide ? 64 : 128) || (few <= (wide ? 400 : 800) && seen <= kWindowShort)) return 16;
  constexpr int32_t one = 16 * kAttnWaves;
  return wide || (rows + 2 * one - 1) / (2 * one) * heads < 256 ? one : 2 * one;
}

// Short windows are as long as one another, so there is nothing to even out where the
// workgroups fill the chip, and a join to save: few rows are not split from one
// workgroup a CU on, more from two.  Longer ones leave CUs idle, whose sequences are
// shorter or which hold a workgroup less than others: few rows that see 4096 tokens are
// split as without a window, with seven eighths of two workgroups a CU and more those
// that see 8192.  us, whole / so, of uneven sequences of up to 12000 or (*) 32768:
//   workgroups [256], D = 128: window 2048 20.7 / 21.9, 4096 30.9 / 30.7, 11000 64.8 / 57.0
//     [320], D = 64: 2048 19.5 / 19.9, 4096 30.0 / 26.9, 8000 49.6 / 40.6, 20000* 121 / 73
//     [320] of 16 rows, D = 64: 4096* 34.6 / 30.3, 20000* 137 / 83
//     [384], D = 128: 2048 28.2 / 29.6, 4096 45.0 / 46.6, 6000 60.2 / 58.1, 11000 88 / 78
//     [480], D = 128: 2048 29.3 / 35.3, 5000 55.0 / 59.7, 8000 86.2 / 85.6
//     [512], D = 128: 8000* 108 / 112, 20000* 218 / 217, 32000* 269 / 254; D = 64: 11000
//       56.9 / 52.9, 32000* 164 / 148
//     [800], D = 64: 8000* 105 / 94, 32000* 247 / 234
//     [1024], D = 64: 4096 52.5 / 57.2, 6000 76 / 81, 11000 115 / 110
// and of equal ones [256], D = 128: 5000 33.8 / 36.1, 8000 51.8 / 53.2; [384], D = 64: 4096
// 30.3 / 27.4, 8000 51 / 43; [512], D = 128: 8000* 117 / 124, 32000* 401 / 403; [800],
// D = 64: 12000* 161 / 146.
// More rows, below two workgroups a CU: the number of splits with the
// least time by what was measured of many rows: a step of a block takes longer the more
// workgroups a CU has (D = 64: 0.75, 0.9, 1.05, 1.2 us with one to four, which is what
// the registers hold; eight waves, two; D = 128, three), and a join 3.5 us and what its
// shares take to write and read.  Of 31 cases (32 to 1000 tokens, windows of 256 to
// 4096, 16 to 376 workgroups, 1 to 16 splits) that is the best in 21 and 1.014 of it in
// the mean (rounded up to whole blocks a split 26 and 1.007, but then a longer window
// may take fewer splits, and the workspace is to grow with it).  us, here / as without
// a window: 512 tokens, D = 64, windows of 512, 1000, 4096 19.0 / 20.6, 28.7 / 26.9,
// 52.2 / 64.1; 256, 4096 32.5 / 38.9; 1000, 1000 28.0 / 35.0; D = 128, 512 tokens, 256
// and 4096 16.4 / 22.2 and 64.6 / 79.7.
int32_t kv4_attn_window_splits(int32_t tile_rows, int64_t workgroups, int64_t max_seen, int head_dim) {
  const bool few = tile_rows <= 16;
  if (few) {
    const bool whole = workgroups >= 256 && max_seen < (workgroups < 448 ? 4096 : 8192);
    return whole ? 1 : kv4_attn_splits(tile_rows, workgroups, max_seen);
  }
  if (workgroups >= 512) return 1;
  const bool eight = tile_rows == 32 * kAttnWaves;
  const int64_t fit = eight ? 512 : head_dim == 64 ? 1024 : 768;
  const int64_t first = head_dim == 64 && !eight ? 600 : 400, more = eight ? 200 : head_dim == 64 ? 150 : 250;  // ns
  const int64_t blocks = max_seen / kKv4Block + 2;
  // times n, exact: a / n + join
  int64_t best = 0, best_a = 0, best_join = 0;
  for (int64_t n = 1; n == 1 || (n * workgroups <= fit && 2 * n <= blocks); n += 1 + n / 16) {
    const int64_t total = n * workgroups;
    const int64_t a = blocks * (first + more * ((total + 255) / 256));
    const int64_t join = n == 1 ? 0 : 3500 + total * tile_rows * head_dim / 800;
    if (best == 0 || (a + join * n) * best < (best_a + best_join * best) * n) best = n, best_a = a, best_join = join;
  }
  return static_cast<int32_t>(best);
}

hipError_t launch_kv4_attn(const AttnArgs& a, int head_dim, int dt, hipStream_t stream) {
  auto go = [&](auto win) {
    constexpr bool kWin = decltype(win)::value;
    if (head_dim == 64)
      return dt == kActF16 ? launch_d<64, kActF16, kWin>(a, stream) : launch_d<64, kActBf16, kWin>(a, stream);
    return dt == kActF16 ? launch_d<128, kActF16, kWin>(a, stream) : launch_d<128, kActBf16, kWin>(a, stream);
  };
  return a.window > 0 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace sherry
