"""How exact attention with a window is where scores are large (fp32 has them only to
units and more), by what holds for any size of them:

  equal keys   weigh the same wherever they lie: a row's result is the mean of the V
               that it sees.  Each weight enters the second product rounded to half a
               step of fp16 (2^-11 of its V scale's share s |c - 7.5|), the sums are
               fp32's (2^-24 a step, of fewer than 2^4 steps of any one sum tree
               beside the tokens' own, L / 32 + 64 of them), the result is rounded once.
  large scores where no other token comes within `size` 2^-19 + 40 of the best one, it
               has all the weight: tests/test_attn_precision.py has the reasons.
"""
import numpy as np
import pytest
import torch

from oracle import layer_ref
from tests.test_attn_gpu import DEV, HALF, host, make_kv, randn, say
from tests.test_attn_precision import SCORE, parts

pytestmark = pytest.mark.gpu

# qs, ls, bound, hq, hkv, d, window, sinks: the kernel that shares out the tokens (one
# token, a few, split; few rows of many tiles), and many rows on eight waves, four, split
CASES = [([1], [900], 900, 4, 1, 64, 700, 4), ([3, 2], [40, 600], 600, 6, 2, 128, 300, 0), ([40], [500], 500, 4, 2, 64, 200, 4),
         ([1100], [1400], 1400, 32, 8, 64, 600, 4), ([300], [2900], 2900, 8, 2, 64, 2700, 4), ([300], [2900], 2900, 8, 2, 128, 2700, 0),
         ([1500], [1600], 1600, 24, 8, 128, 500, 20), ([300], [2900], 2900, 8, 2, 64, 2800, 200)]


class Seqs:
    """Sequences on pages in order; q and k of chosen sizes."""

    def __init__(self, lib, qs, ls, bound, hq, hkv, d, window, sinks, dtype, seed, q_power=0, key=None):
        page = 64
        need = [-(-length // page) for length in ls]
        self.cache = lib.Kv4Cache(sum(need), page, hkv, d)
        first = np.concatenate([[0], np.cumsum(need)])
        table = np.zeros((len(ls), max(need)), np.int32)
        self.kp, self.vp = [], []
        for i, length in enumerate(ls):
            table[i, :need[i]] = np.arange(first[i], first[i + 1])
            k, v = make_kv(length, hkv, d, dtype, seed + 10 * i + 1)
            if key is not None:
                k = key(k)
            lib.kv4_write(self.cache, k.to(DEV), v.to(DEV), torch.arange(length, device=DEV) + int(first[i]) * page)
            self.kp.append(parts(k))
            self.vp.append(parts(v))
        self.q = (randn(sum(qs), hq, d, seed=seed) * 2.0 ** q_power).to(dtype)
        self.lib, self.qs, self.ls, self.window, self.sinks, self.scale = lib, qs, ls, window, sinks, d ** -0.5
        self.args = (torch.from_numpy(table).to(DEV), torch.tensor(ls, dtype=torch.int32, device=DEV))
        self.kw = dict(cu_q=torch.tensor(np.concatenate([[0], np.cumsum(qs)]), dtype=torch.int32, device=DEV), max_q=max(qs),
                       max_kv=bound, want_lse=True, scale=self.scale, window=window, sinks=sinks)

    def run(self):
        out, lse = self.lib.kv4_attn(self.cache, self.q.to(DEV), *self.args, **self.kw)
        torch.cuda.synchronize()
        return host(out).astype(np.float64), host(lse).astype(np.float64)

    def rows(self, every=1):
        """sequence, row of q, place among the sequence's new tokens"""
        at = 0
        for i, n in enumerate(self.qs):
            for r in range(0, n, every):
                yield i, at + r, r
            at += n

    def seen(self, i, r):
        return np.flatnonzero(layer_ref.visible(self.qs[i], self.ls[i], self.window, self.sinks)[r])


@pytest.mark.parametrize("qs,ls,bound,hq,hkv,d,window,sinks", CASES)
@pytest.mark.parametrize("dtype,q_power,constant", [(torch.bfloat16, 0, False), (torch.float16, 6, True), (torch.bfloat16, 20, True),
                                                    (torch.bfloat16, 20, False), (torch.bfloat16, 27, False), (torch.bfloat16, 60, True)])
def test_equal_keys_weigh_the_same(gpu_lib, qs, ls, bound, hq, hkv, d, window, sinks, dtype, q_power, constant):
    say("window equal keys", qs, ls, hq, hkv, d, window, sinks, dtype, q_power, constant)

    def same(k):
        one = k[:1].float()
        if constant:
            one = one.new_full(one.shape, -1.37)  # (a scale of 0: the zero point is the score)
        return one.expand(k.shape).to(dtype).contiguous()
    b = Seqs(gpu_lib, qs, ls, bound, hq, hkv, d, window, sinks, dtype, 3000 + d, q_power, same)
    out, lse = b.run()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    for i, row, r in b.rows(7):
        at = b.seen(i, r)
        q = host(b.q[row]).astype(np.float64)
        for h in range(hq):
            kh = h // (hq // hkv)
            v, vr, vp = (b.vp[i][j][at, kh] for j in (0, 2, 1))
            ref = v.mean(0)
            tol = HALF[dtype] * np.abs(ref) + 2.0 ** -11 * vr.mean(0) + (len(at) / 32 + 80) * 2.0 ** -24 * vp.mean(0)
            off = np.abs(out[row, h] - ref)
            assert (off <= tol).all(), (row, h, off.max(), tol.max())
            s = b.scale * (b.kp[i][0][at[0], kh] @ q[h])
            size = abs(b.scale) * (np.abs(q[h]) @ b.kp[i][1][at[0], kh])
            want = s + np.log(len(at))
            assert abs(lse[row, h] - want) <= 2.0 ** -20 + SCORE * size + 2.0 ** -22 * abs(want), (row, h)


@pytest.mark.parametrize("qs,ls,bound,hq,hkv,d,window,sinks", CASES)
@pytest.mark.parametrize("q_power", [14, 20, 25, 31, 60])
def test_large_scores_are_one_token(gpu_lib, qs, ls, bound, hq, hkv, d, window, sinks, q_power):
    dtype = torch.bfloat16
    say("window large scores", qs, ls, hq, hkv, d, window, sinks, q_power)
    b = Seqs(gpu_lib, qs, ls, bound, hq, hkv, d, window, sinks, dtype, 3100 + d, q_power)
    out, lse = b.run()
    told = 0
    for i, row, r in b.rows(7):
        at = b.seen(i, r)
        q = host(b.q[row]).astype(np.float64)
        for h in range(hq):
            kh = h // (hq // hkv)
            s = b.scale * (b.kp[i][0][at, kh] @ q[h])
            size = abs(b.scale) * (np.abs(q[h]) @ b.kp[i][1][at, kh].T).max()
            assert abs(lse[row, h] - s.max()) <= 2.0 ** -20 + SCORE * size + 2.0 ** -22 * abs(s.max()) + np.log(len(at))
            v = b.vp[i][0][at, kh]
            first, second = np.sort(s)[::-1][:2]
            lo, hi = v.min(0), v.max(0)
            if first - second > 2 * SCORE * size + 40:
                told += 1
                lo = hi = v[s.argmax()]
            tol = 2.0 ** -11 * b.vp[i][2][at, kh].max(0) + np.maximum(np.abs(lo), np.abs(hi)) * HALF[dtype] + \
                2.0 ** -20 * b.vp[i][1][at, kh].max(0)
            assert (out[row, h] >= lo - tol).all() and (out[row, h] <= hi + tol).all(), (row, h)
    say(f"   {told} rows are one token")
    assert told
