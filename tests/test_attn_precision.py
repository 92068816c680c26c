"""How exact attention over the 4-bit cache is, by bounds that follow each row's
own sizes (tests/test_attn_gpu.py bounds every row by the largest one).

With codes c, scale s and zero point z of a value, w a row's softmax weights:
  score   `size` = scale * max over the row's tokens of sum_d |q_d| (15 s + |z|).
          A query element enters the matrix core as it is or to 2^-36 of the row's
          largest; of few rows, K's codes enter with up to six leading zeros, whose
          sums the core cuts by as many bits: 2^-17 of s |q| a term in the worst
          case, 2^-18.8 as the root mean square of a uniform cut.  64 of them as a
          random sum: 2^-15.8 s max|q|, where sum |q| 15 s is about 2^8 s max|q| or
          more.  2^-23.8 of `size`, so 2^-20 leaves it a factor of 14 for its
          tails, D = 128 and other rows; of many log-sums the root mean square may
          be twice 2^-23.8.  A log-sum's own steps (sums of up to L / 32 + 64
          tokens, a logarithm, a product) are 2^-22 of 1 + itself likewise.
  weight  P = p s is rounded to fp16 in the second product: half a step, 2^-11 at
          mantissa 1, is 2^-11 / sqrt(3) as a root mean square and with mantissas
          spread evenly over their logarithm (mean of 1 / m^2 over [1, 2): 0.541)
          0.425 * 2^-11 of each term w s |c - 7.5|.
  result  rounded once; its own rounding is taken from the exact result.
"""
import numpy as np
import pytest
import torch

from oracle import attn_ref
from tests.test_attn_gpu import DEV, HALF, Batch, gen, host, make_kv, randn, say

P_RMS = 0.425 * 2.0 ** -11
SCORE, SCORE_RMS = 2.0 ** -20, 2.0 ** -23.8


def parts(x):
    """value, 15 s + |z| and s |c - 7.5| of what the cache holds of x"""
    c, s, z = attn_ref.quantise(host(x))
    g = c.shape[:-1] + (c.shape[-1] // 64, 64)
    s64 = np.broadcast_to(s.astype(np.float64)[..., None], g)
    z64 = np.broadcast_to(np.abs(z.astype(np.float64))[..., None], g)
    return (attn_ref.dequantise(c, s, z), (15 * s64 + z64).reshape(c.shape),
            (s64 * np.abs(c.reshape(g) - 7.5)).reshape(c.shape))


@np.errstate(invalid="ignore")  # (spoiled rows)
def exact(q, k, v, scale):
    """out, lse, size [n, hq] and what the weights' rounding and the scores' error
    make of a result as a root mean square [n, hq, d] each, in fp64; k and v from
    parts()."""
    n, hq, d = q.shape
    length, hkv = k[0].shape[:2]
    out, var, svar = (np.zeros((n, hq, d)) for _ in range(3))
    lse, size = np.full((n, hq), -np.inf), np.zeros((n, hq))
    seen = np.arange(length)[None, :] <= np.arange(n)[:, None] + length - n
    for h in range(hq if length else 0):
        kh = h // (hq // hkv)
        s = np.where(seen, scale * (q[:, h] @ k[0][:, kh].T), -np.inf)
        size[:, h] = abs(scale) * np.where(seen, np.abs(q[:, h]) @ k[1][:, kh].T, 0).max(-1)
        live = seen.any(-1)
        m = np.where(live, s.max(-1), 0)
        e = np.exp(s - m[:, None])
        total = np.where(live, e.sum(-1), 1)
        lse[live, h] = (m + np.log(total))[live]
        w = e / total[:, None]
        out[:, h] = w @ v[0][:, kh]
        w2, o, x = w * w, out[:, h], v[0][:, kh]
        var[:, h] = w2 @ (v[2][:, kh] ** 2)
        svar[:, h] = w2 @ (x * x) - 2 * o * (w2 @ x) + o * o * w2.sum(-1, keepdims=True)
    return out, lse, size, P_RMS * np.sqrt(var), SCORE_RMS * size[..., None] * np.sqrt(np.maximum(svar, 0))


def rounded(x, dtype):
    return torch.from_numpy(x).to(dtype).double().numpy()


def check(q, k, v, scale, out, lse, dtype, keep=None, weight_bits=True):
    """Norm of the results' error against their own rounding and P's; every
    log-sum against its row's size.  keep [n, hq]: rows that are looked at."""
    ref, rl, size, p, ps = exact(q, k, v, scale)
    keep = np.ones(q.shape[:2], bool) if keep is None else keep
    empty = np.isneginf(rl)
    assert not out[empty & keep].any() and np.isneginf(lse[empty & keep]).all()
    keep = keep & ~empty
    if not keep.any():
        return
    assert np.isfinite(out[keep]).all() and np.isfinite(lse[keep]).all()
    lerr = np.abs(lse[keep] - rl[keep])
    lmax = (lerr / (2.0 ** -20 + SCORE * size[keep] + 2.0 ** -22 * np.abs(rl[keep]))).max()
    lrms = np.sqrt(((lerr / (SCORE_RMS * size[keep] + 2.0 ** -22 * (1 + np.abs(rl[keep])))) ** 2).mean())
    err = np.linalg.norm((out - ref)[keep])
    own = np.linalg.norm([np.linalg.norm(x[keep]) for x in (rounded(ref, dtype) - ref, weight_bits * p, ps)])
    say(f"   log-sum {lmax:.3f} of its bound, {lrms:.3f} of its rounding, result {err / own:.3f}")
    assert lmax <= 1 and lrms <= 2 and err <= 1.25 * own


class Rows(Batch):
    def check_rows(self, out, lse, keep=None, weight_bits=True):
        at = 0
        for i, n in enumerate(self.qs):
            if n:
                k, v = ([a for a in x[i]] for x in (self.kp, self.vp))
                f = slice(at, at + n)
                check(host(self.q[f]).astype(np.float64), k, v, self.scale, host(out[f]).astype(np.float64),
                      host(lse[f]).astype(np.float64), self.dtype, None if keep is None else keep[f], weight_bits)
            at += n

    def __init__(self, lib, qs, ls, hq, hkv, d, page_size, dtype, seed, **kw):
        super().__init__(lib, qs, ls, hq, hkv, d, page_size, dtype, seed, **kw)
        self.kp, self.vp = [], []
        for i, length in enumerate(ls):
            k, v = make_kv(length, hkv, d, dtype, seed + 10 * i + 1) if length else (torch.zeros(0, hkv, d),) * 2
            self.kp.append(parts(k))
            self.vp.append(parts(v))
        self.page_size, self.made = page_size, lambda i: make_kv(ls[i], hkv, d, dtype, seed + 10 * i + 1)

    def write(self, i, change):
        """Sequence i's keys and values again, as `change` makes them of what they were."""
        k, v = change(*self.made(i))
        j = torch.arange(len(k), device=DEV)
        slots = self.table[i].long()[j // self.page_size] * self.page_size + j % self.page_size
        self.lib.kv4_write(self.cache, k.to(DEV), v.to(DEV), slots)
        self.kp[i], self.vp[i] = parts(k), parts(v)


def made(dtype, n=40, length=300, hq=4, hkv=2, d=64, seed=2700, q_scale=1.0, q_noise=0.0, p_bits=11):
    """Attention in fp64 with P rounded to p_bits and q off by q_noise of itself:
    what check() is given of it."""
    k, v = (parts(x) for x in make_kv(length, hkv, d, dtype, seed))
    q = host((randn(n, hq, d, seed=seed + 5) * q_scale).to(dtype)).astype(np.float64)
    used = q * (1 + q_noise * np.random.default_rng(seed).uniform(-1, 1, q.shape))
    out, lse = exact(used, k, v, d ** -0.5)[:2]
    seen = np.arange(length)[None, :] <= np.arange(n)[:, None] + length - n
    for h in range(hq):
        kh = h // (hq // hkv)
        w = np.where(seen, np.exp(d ** -0.5 * (used[:, h] @ k[0][:, kh].T) - lse[:, [h]]), 0)
        m, e = np.frexp(w)
        out[:, h] += (np.ldexp(np.rint(m * 2.0 ** p_bits), e - p_bits) - w) @ (np.sign(v[0][:, kh]) * v[2][:, kh])
    return q, k, v, d ** -0.5, rounded(out, dtype), lse, dtype


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kw", [{}, dict(d=128, n=33, hq=10), dict(length=1000), dict(q_scale=30.0)])
def test_bounds_tell_mistakes(dtype, kw):
    """The bounds hold for 11 bits of P and exact scores, and neither for 8 bits
    nor for queries that are 2^-11 off (no GPU: computed here)."""
    check(*made(dtype, **kw))
    for mistake in (dict(p_bits=8), dict(q_noise=2.0 ** -11)):
        if kw.get("q_scale") and "p_bits" in mistake:
            continue  # (few tokens have the weight, whose rounding is a smaller part)
        with pytest.raises(AssertionError):
            check(*made(dtype, **kw, **mistake))


# more than 16 rows a key head, on each tile of the many-row rule (its bound of lengths picks the tile)
MANY = [([40], [300], 300, 4, 2, 64), ([33, 70], [310, 90], 310, 10, 5, 128),
        ([100, 129], [300, 290], 2100, 40, 10, 64), ([140], [300], 4000, 176, 176, 64),
        ([140], [300], 4000, 176, 176, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("qs,ls,bound,hq,hkv,d", MANY)
@pytest.mark.parametrize("power", [14, 28, 36, 60, -30])
def test_one_row_of_another_size(gpu_lib, qs, ls, bound, hq, hkv, d, power):
    """One bf16 row 2^power times its neighbours leaves them as exact as ever."""
    say("attn mixed sizes", qs, ls, bound, hq, hkv, d, power)
    b = Rows(gpu_lib, qs, ls, hq, hkv, d, 64, torch.bfloat16, 2000 + d)
    b.q[7, 1] *= 2.0 ** power
    keep = np.ones(b.q.shape[:2], bool)
    keep[7, 1] = power < 0  # (the large one's scores are past any bound of use)
    out, lse = b.run(max_kv=bound)
    b.check_rows(out, lse, keep)


@pytest.mark.gpu
def test_fp16_rows_of_other_sizes(gpu_lib):
    """fp16 rows at both ends of the type's range in one tile."""
    say("attn mixed sizes fp16")
    b = Rows(gpu_lib, [40], [300], 4, 2, 64, 64, torch.float16, 2100)
    b.q[3] *= 2.0 ** 13
    b.q[4] *= 2.0 ** -12
    keep = np.ones(b.q.shape[:2], bool)
    keep[3] = False
    out, lse = b.run()
    b.check_rows(out, lse, keep)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", [2.0 ** 50, 2.0 ** 126, float("inf"), float("nan")])
def test_padding_rows_hold_anything(gpu_lib, d, what):
    """Rows that see nothing (more new tokens than cached ones) may hold any
    bits: they give zeros, and their neighbours what they give without them."""
    say("attn padding rows", d, what)
    b = Rows(gpu_lib, [50, 50], [20, 37], 4, 2, d, 32, torch.bfloat16, 2200)
    b.q[:30] = what
    b.q[50:63] = -what
    b.check_rows(*b.run())


@pytest.mark.gpu
@pytest.mark.parametrize("qs,ls,bound,hq,hkv,d", MANY)
def test_spoiled_rows_stay_alone(gpu_lib, qs, ls, bound, hq, hkv, d):
    """NaN, infinity and a size past the contract (|scale q| < 2^90) in single
    rows of a tile of many."""
    say("attn spoiled rows", qs, ls, bound, hq, hkv, d)
    b = Rows(gpu_lib, qs, ls, hq, hkv, d, 64, torch.bfloat16, 2300 + d)
    keep = np.ones(b.q.shape[:2], bool)
    for row, head, what in ((5, 0, float("nan")), (6, 1, float("inf")), (9, 0, -float("inf")), (11, 1, 2.0 ** 125)):
        b.q[row, head, 3] = what
        keep[row, head] = False
    out, lse = b.run(max_kv=bound)
    b.check_rows(out, lse, keep)
    assert torch.isnan(out[5, 0]).all() and not torch.isfinite(out[6, 1]).all()


# the few-row kernel (one token, a few, many splits) and the many-row one
LARGE = [([1], [200], 200, 4, 1, 64), ([3, 2], [40, 300], 300, 6, 2, 128), ([1, 1], [5000, 40], 5000, 8, 2, 64),
         ([40], [300], 300, 4, 2, 64), ([33, 70], [310, 90], 310, 10, 5, 128), ([40], [900], 100000, 4, 2, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("qs,ls,bound,hq,hkv,d", LARGE)
@pytest.mark.parametrize("dtype,q_power,k_power", [
    (torch.bfloat16, 14, 0), (torch.bfloat16, 20, 0), (torch.bfloat16, 25, 0), (torch.bfloat16, 31, 0),
    (torch.bfloat16, 60, 0), (torch.bfloat16, 60, 10), (torch.float16, 12, 0), (torch.float16, 13, 11)])
def test_large_scores(gpu_lib, qs, ls, bound, hq, hkv, d, dtype, q_power, k_power):
    """Scores up to 2^80, where the softmax is one token unless two are closer
    than fp32 can tell (`size` 2^-20, at both ends of the difference): that
    token's values to their rounding and P's, else something between the values."""
    say("attn large scores", qs, ls, bound, hq, hkv, d, dtype, q_power, k_power)
    b = Rows(gpu_lib, qs, ls, hq, hkv, d, 64, dtype, 2400 + d, q_scale=2.0 ** q_power)
    for i in range(len(ls)):
        b.write(i, lambda k, v: ((k.float() * 2.0 ** k_power).to(k.dtype), v))
    out, lse = b.run(max_kv=bound)
    at = told = 0
    for i, n in enumerate(qs):
        q = host(b.q[at:at + n]).astype(np.float64)
        got, gl = (host(x[at:at + n]).astype(np.float64) for x in (out, lse))
        _, rl, size = exact(q, b.kp[i], b.vp[i], b.scale)[:3]
        assert (np.abs(gl - rl) <= 2.0 ** -20 + SCORE * size + 2.0 ** -22 * np.abs(rl)).all()
        for r in range(n):
            for h in range(hq):
                kh = h // (hq // hkv)
                seen = ls[i] - n + r + 1
                s = b.scale * (b.kp[i][0][:seen, kh] @ q[r, h])
                v, pv = b.vp[i][0][:seen, kh], 2.0 ** -11 * b.vp[i][2][:seen, kh].max(0)
                first, second = np.sort(s)[::-1][:2] if seen > 1 else (s[0], -np.inf)
                lo, hi = v.min(0), v.max(0)
                if first - second > 2 * SCORE * size[r, h] + 40:  # (e^-40 of the others is nothing)
                    told += 1
                    lo = hi = v[s.argmax()]
                tol = pv + np.maximum(np.abs(lo), np.abs(hi)) * HALF[dtype] + 2.0 ** -20 * b.vp[i][1][:seen, kh].max(0)
                assert (got[r, h] >= lo - tol).all() and (got[r, h] <= hi + tol).all(), (r, h)
        at += n
    say(f"   {told} of {sum(qs) * hq} rows are one token")
    assert told


@pytest.mark.gpu
@pytest.mark.parametrize("qs,ls,bound,hq,hkv,d", LARGE)
def test_every_score_far_below_zero(gpu_lib, qs, ls, bound, hq, hkv, d):
    """Scores of -2^106 and less on every token (exact ties among them, of exact
    keys): no row takes them for nothing seen, in a wave, a share or a join."""
    say("attn negative scores", qs, ls, bound, hq, hkv, d)
    b = Rows(gpu_lib, qs, ls, hq, hkv, d, 64, torch.bfloat16, 2500 + d)
    b.q = torch.full_like(b.q, 2.0 ** 92)
    for i, length in enumerate(ls):
        b.write(i, lambda k, v: ((-2000.0 - torch.arange(length) % 40).view(-1, 1, 1).expand(k.shape).half(), v.half()))
    b.check_rows(*b.run(max_kv=bound))


@pytest.mark.gpu
@pytest.mark.parametrize("qs,ls", [([5], [9]), ([1, 4, 2], [30, 4, 70]), ([40, 3], [300, 3])])
def test_ragged_call_without_max_q(gpu_lib, qs, ls):
    """Every row of every sequence is computed, and rows of none are zeros."""
    say("attn cu_q without max_q", qs, ls)
    b = Rows(gpu_lib, qs, ls, 4, 2, 64, 64, torch.float16, 2600)
    b.q = torch.cat([b.q, b.q[:3]])
    junk = [torch.full_like(b.q, 7.0, device=DEV) for _ in range(4)]  # (what a fresh buffer would hold)
    del junk
    out, lse = b.lib.kv4_attn(b.cache, b.q.to(DEV), b.table, b.lens, cu_q=b.cu, want_lse=True)
    b.check_rows(out, lse)
    assert not out[sum(qs):].any() and torch.isneginf(lse[sum(qs):]).all()


FEW = [([1] * 4, [1, 40, 200, 1031], 1031, 4, 1, 64), ([5, 1, 7], [5, 77, 300], 300, 6, 2, 128),
       ([1, 1], [9001, 20], 9001, 8, 2, 64), ([4, 4], [4099, 700], 4099, 4, 4, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("qs,ls,bound,hq,hkv,d", FEW + MANY + [([500], [4000], 4000, 8, 2, 64)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("q_scale", [1.0, 30.0])
def test_results_to_their_rounding(gpu_lib, qs, ls, bound, hq, hkv, d, dtype, q_scale):
    """Results carry their own rounding and P's (of up to 16 fp16 rows their own
    alone), log-sums fp32's."""
    say("attn precision", qs, ls, bound, hq, hkv, d, dtype, q_scale)
    b = Rows(gpu_lib, qs, ls, hq, hkv, d, 64, dtype, 2800 + d, q_scale=q_scale)
    b.check_rows(*b.run(max_kv=bound), weight_bits=dtype == torch.bfloat16 or max(qs) * hq // hkv > 16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("qs,ls,hq,hkv,d", [([1, 1], [9001, 20], 8, 2, 64), ([3], [4000], 4, 2, 128), ([64], [3000], 4, 1, 64)])
def test_splits_change_a_rounding_step(gpu_lib, qs, ls, hq, hkv, d, dtype):
    """Any number of splits gives the same results up to a step of the result's
    type, and mostly the same bits: P's rounding (its own in every split) moves a
    value by under 2^-11 of its terms, their sum over L tokens by less."""
    say("attn splits", qs, ls, hq, hkv, d, dtype)
    b = Rows(gpu_lib, qs, ls, hq, hkv, d, 64, dtype, 2900 + d)
    outs = []
    for max_kv in (0, 600, 1200, max(ls), 1 << 30):
        o, lse = b.run(max_kv=max_kv)
        b.check_rows(o, lse, weight_bits=dtype == torch.bfloat16 or max(qs) * hq // hkv > 16)
        outs.append(host(o).astype(np.float64))
    one = outs[0]
    for o in outs[1:]:
        step = 2 * HALF[dtype] * np.maximum(np.abs(o), np.abs(one))
        assert (np.abs(o - one) <= step + 2.0 ** -11 * max(x[2].max() for x in b.vp)).all()
        assert np.linalg.norm(o - one) <= np.linalg.norm(step)
