"""Attention operators on the GPU at sizes that choose other variants of their
kernels: several heads a lane, outputs past the caches, and bounds of the new
tokens that cut a sequence."""
import numpy as np
import pytest
import torch

from oracle import attn_ref
from tests.test_attn_gpu import DEV, Batch, gen, host, make_kv, randn, rope_tolerance, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,hq,hkv,d,rot,inter", [(33000, 1, 1, 64, 32, False), (9001, 7, 1, 128, 128, True),
                                                  (9000, 5, 3, 112, 48, False)])
@pytest.mark.parametrize("norms", ["q", "k"])
def test_rope_many_tokens(gpu_lib, n, hq, hkv, d, rot, inter, norms):
    """Four heads a lane, counts that are no multiple of it, and the norm on one
    side only: lanes of one wave with and without it."""
    say("rope many tokens", n, hq, hkv, d, rot, inter, norms)
    x = randn(n, hq + hkv, d, seed=n, dtype=torch.bfloat16)
    ang = np.random.default_rng(n).uniform(-7, 7, (500, rot // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    pos = torch.randint(0, 500, (n,), generator=gen(n + 1))
    w = 1 + 0.3 * randn(d, seed=n + 2)
    wq, wk = (w if norms == s else None for s in "qk")
    g = x.to(DEV)
    ys = gpu_lib.qk_norm_rope(g[:, :hq], g[:, hq:], torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV),
                              pos.to(DEV), q_weight=None if wq is None else wq.to(DEV),
                              k_weight=None if wk is None else wk.to(DEV), eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    c, s = cos[pos.numpy()], sin[pos.numpy()]
    for part, weight, y in ((x[:, :hq], wq, ys[0]), (x[:, hq:], wk, ys[1])):
        args = (host(part), None if weight is None else weight.numpy(), c, s, 1e-5, rot, inter)
        tol = rope_tolerance(*args, torch.bfloat16)
        assert (np.abs(host(y).astype(np.float64) - attn_ref.norm_rope(*args)) <= tol).all()


def test_kv4_read_past_the_caches(gpu_lib):
    """A read whose outputs are stored past the caches gives what small ones give."""
    say("kv4 read many")
    n, heads, d = 20011, 8, 64
    cache = gpu_lib.Kv4Cache(-(-n // 64) + 1, 64, heads, d)
    k, v = make_kv(n, heads, d, torch.float16, 50)
    slots = torch.arange(n, device=DEV) + 37
    gpu_lib.kv4_write(cache, k.to(DEV), v.to(DEV), slots)
    rk, rv = gpu_lib.kv4_read(cache, slots)
    for a in range(0, n, 1999):
        pk, pv = gpu_lib.kv4_read(cache, slots[a:a + 1999])
        assert torch.equal(rk[a:a + 1999], pk) and torch.equal(rv[a:a + 1999], pv)
    want = attn_ref.dequantise(*attn_ref.quantise(host(k[:500])))
    assert (np.abs(host(rk[:500]).astype(np.float64) - want) <= np.abs(want) * 2.0 ** -11 * (1 + 2.0 ** -12) + 2.0 ** -25).all()


@pytest.mark.parametrize("qs,ls,max_q", [([5, 2], [40, 9], 3), ([70, 40], [90, 300], 33), ([4], [9000], 2)])
def test_attn_max_q_cuts_a_sequence(gpu_lib, qs, ls, max_q):
    """Of a sequence of more new tokens than max_q the first max_q rows are
    computed, at their own places in the sequence; the others stay as they were."""
    say("attn max_q cuts", qs, ls, max_q)
    b = Batch(gpu_lib, qs, ls, 4, 2, 64, 64, torch.float16, 3100)
    whole, lse = b.run()
    b.check(whole, lse)
    out, l2 = torch.full_like(whole, 9.0), torch.full_like(lse, 9.0)
    b.run(max_q=max_q, out=out, lse=l2)
    torch.cuda.synchronize()
    at = 0
    for n in qs:
        cut = min(n, max_q)
        b_out, w_out = (host(x[at:at + cut]).astype(np.float64) for x in (out, whole))
        assert (np.abs(b_out - w_out) <= 2.0 ** -10 * (np.abs(w_out) + 1)).all()  # (both within their rounding)
        assert (out[at + cut:at + n] == 9).all() and (l2[at + cut:at + n] == 9).all()
        at += n
