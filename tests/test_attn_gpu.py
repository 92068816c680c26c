"""Attention operators on the GPU against the CPU reference (oracle/attn_ref.py).

Tolerances, from the number formats (half a step: fp16 2^-11, bf16 2^-8, fp32
2^-24 of the value):
  cache: codes and scales bit for bit; values read back one fp32 step and one
    rounding to the output type.
  rotation: fp32 throughout; see rope_tolerance().
  attention: the weights enter the product as fp16 P = p s, beside the exact
    codes: each term is off by at most 2^-11 of p s |c - mid|, |c - mid| <=
    |c - 7.5| + 0.5.  A score (in natural units) is off by at most `ds`, which
    moves a weight by the factor e^(+-2 ds).  The result is rounded once.  See
    attn_reference().
"""
import numpy as np
import pytest
import torch

from oracle import attn_ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0, torch.float32: 0.0}  # half a subnormal step


def say(*a):
    print(*a, flush=True)


def host(t):
    return t.detach().cpu().float().numpy() if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=gen(seed)).to(dtype)


# -------------------------------------------------------------- rotation ---

def rope_tolerance(x, w, cos, sin, eps, rot, inter, out_dtype):
    """fp32 error of y = a c - b s: each factor carries at most 8 half steps
    (mean of up to 256 squares summed over 16 lanes of 16: 20 additions and a
    square each, halved by the root; root, quotient and two products), the
    products and their difference three more: 24 half steps of |a c| + |b s|."""
    mag = attn_ref.norm_rope(np.abs(x), w if w is None else np.abs(w), np.abs(cos), -np.abs(sin), eps, rot, inter)
    mag = np.abs(mag)
    # |a c| + |b s| for the first of a pair, |b c| + |a s| for the second
    other = attn_ref.norm_rope(np.abs(x), w if w is None else np.abs(w), np.abs(cos), np.abs(sin), eps, rot, inter)
    mag = np.maximum(mag, np.abs(other))
    return 24 * 2.0 ** -24 * mag * (1 + HALF[out_dtype]) + mag * HALF[out_dtype] + TINY[out_dtype]


def check_rope(gpu_lib, n, hq, hkv, d, rot, inter, norm, x_dt, y_dt, seed, maxpos=500, in_place=False):
    qkv = randn(n, (hq + 2 * hkv) * d, seed=seed, dtype=x_dt).to(DEV)
    q = qkv[:, :hq * d].view(n, hq, d)
    k = qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
    v_before = qkv[:, (hq + hkv) * d:].clone()
    xq, xk = host(q).copy(), host(k).copy()
    ang = np.random.default_rng(seed).uniform(-7, 7, (maxpos, rot // 2))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    pos = torch.randint(0, maxpos, (n,), generator=gen(seed + 1))
    wq = (1 + 0.3 * randn(d, seed=seed + 2)) if norm else None
    wk = (1 + 0.3 * randn(d, seed=seed + 3)) if norm else None
    to = lambda a: None if a is None else a.to(DEV)  # noqa: E731
    yq, yk = gpu_lib.qk_norm_rope(q, k, torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV), pos.to(DEV),
                                  q_weight=to(wq), k_weight=to(wk), eps=1e-5, interleaved=inter, out_dtype=y_dt,
                                  q_out=q if in_place else None, k_out=k if in_place else None)
    torch.cuda.synchronize()
    c, s = cos[pos.numpy()], sin[pos.numpy()]
    for x, w, y in ((xq, wq, yq), (xk, wk, yk)):
        w = None if w is None else w.numpy()
        ref = attn_ref.norm_rope(x, w, c, s, 1e-5, rot, inter)
        tol = rope_tolerance(x, w, c, s, 1e-5, rot, inter, y.dtype)
        err = np.abs(host(y).astype(np.float64) - ref)
        assert (err <= tol).all(), (err - tol).max()
    assert torch.equal(qkv[:, (hq + hkv) * d:], v_before)


@pytest.mark.parametrize("n,hq,hkv,d,rot,inter,norm", [
    (1, 32, 8, 64, 64, False, False), (1, 1, 1, 16, 16, True, True), (3, 24, 8, 128, 128, False, True),
    (77, 5, 5, 96, 32, True, True), (130, 4, 2, 80, 48, False, True), (33, 2, 1, 256, 256, False, True),
    (9, 3, 1, 208, 64, True, False), (1000, 7, 1, 64, 32, False, True), (5, 2, 2, 48, 48, True, True)])
@pytest.mark.parametrize("x_dt,y_dt", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                       (torch.float32, torch.float16), (torch.float16, torch.float32)])
def test_rope(gpu_lib, n, hq, hkv, d, rot, inter, norm, x_dt, y_dt):
    say("rope", n, hq, hkv, d, rot, inter, norm, x_dt, y_dt)
    check_rope(gpu_lib, n, hq, hkv, d, rot, inter, norm, x_dt, y_dt, 100 + n)


def test_rope_in_place_and_q_alone(gpu_lib):
    say("rope in place")
    check_rope(gpu_lib, 41, 8, 2, 64, 64, False, True, torch.bfloat16, torch.bfloat16, 7, in_place=True)
    q = randn(5, 3, 64, seed=8, dtype=torch.float16).to(DEV)
    cs = torch.ones(4, 32, device=DEV)
    y, none = gpu_lib.qk_norm_rope(q, None, cs, torch.zeros_like(cs), torch.zeros(5, dtype=torch.int64, device=DEV))
    assert none is None and torch.equal(y, q)
    e, none = gpu_lib.qk_norm_rope(q[:0], None, cs, cs, torch.zeros(0, dtype=torch.int64, device=DEV))
    assert e.shape == (0, 3, 64)


def test_rope_position_out_of_range(gpu_lib):
    """Rotated values of such a token are NaN; other tokens, and the values
    that do not rotate, are as ever."""
    say("rope bad positions")
    q = randn(4, 2, 64, seed=9, dtype=torch.float16).to(DEV)
    cs = torch.ones(10, 16, device=DEV)
    pos = torch.tensor([3, -1, 10, 9], device=DEV)
    y, _ = gpu_lib.qk_norm_rope(q, None, cs, torch.zeros_like(cs), pos)
    torch.cuda.synchronize()
    assert torch.isnan(y[1:3, :, :32]).all() and torch.equal(y[:, :, 32:], q[:, :, 32:])
    assert torch.equal(y[0], q[0]) and torch.equal(y[3], q[3])


def test_rope_zero_and_huge_rows(gpu_lib):
    """A zero head stays zero under the norm (eps), and values whose squares
    still fit fp32 are normalised."""
    say("rope zero and huge")
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    q[0, 1] = 1e18
    cs = torch.ones(1, 32, device=DEV)
    y, _ = gpu_lib.qk_norm_rope(q, None, cs, torch.zeros_like(cs), torch.zeros(1, dtype=torch.int64, device=DEV),
                                q_weight=torch.ones(64, device=DEV))
    assert not y[0, 0].any() and torch.equal(y[0, 1], torch.ones_like(y[0, 1]))


# ----------------------------------------------------------------- cache ---

def make_kv(n, heads, d, dtype, seed):
    k = randn(n, heads, d, seed=seed) * 2 + 3 * randn(1, heads, d, seed=seed + 1)
    v = randn(n, heads, d, seed=seed + 2) * 0.4
    if n > 2:
        k[0, 0, :64] = 1.25           # a constant group: scale 0
        v[1, -1] = 0
        k[2, 0, :64] = torch.arange(64) % 31 * 0.5  # ties: 15 over 15 is 1
    return k.to(dtype), v.to(dtype)


def oracle_cache(cache, k, v, slots, data):
    kq, vq = attn_ref.quantise(host(k)), attn_ref.quantise(host(v))
    for i, slot in enumerate(slots):
        if not 0 <= slot < cache.n_pages * cache.page_size:
            continue
        for h in range(cache.n_kv_heads):
            attn_ref.store(data, cache.page_size, cache.n_kv_heads, int(slot), h, kq[0][i, h], kq[1][i, h], kq[2][i, h],
                           vq[0][i, h], vq[1][i, h], vq[2][i, h])
    return attn_ref.dequantise(*kq), attn_ref.dequantise(*vq)


SLOTS = {
    "one": lambda n, cap, r: r.permutation(cap)[:1],
    "scattered": lambda n, cap, r: r.permutation(cap)[:n],
    "run": lambda n, cap, r: np.arange(n) + 5,
    "aligned run": lambda n, cap, r: np.arange(n) + 32,
    "skips": lambda n, cap, r: np.where(r.random(n) < 0.3, r.choice([-1, cap, cap + 10 ** 12, -2 ** 62], n),
                                        r.permutation(cap)[:n]),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page_size,heads", [(32, 1), (64, 3), (256, 2)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", list(SLOTS))
def test_kv4_write_and_read(gpu_lib, d, page_size, heads, dtype, how):
    """Every byte of the cache, those of other tokens among them, and the values
    read back in each type."""
    say("kv4", d, page_size, heads, dtype, how)
    n_pages = 512 // page_size
    n = 133
    cap = n_pages * page_size
    slots = SLOTS[how](n, cap, np.random.default_rng(d + page_size + heads)).astype(np.int64)
    n = len(slots)
    k, v = make_kv(n, heads, d, dtype, 20 + d)
    cache = gpu_lib.Kv4Cache(n_pages, page_size, heads, d)
    cache.data.fill_(0xA5)
    ref = np.full(cache.nbytes, 0xA5, np.uint8)
    kd, vd = oracle_cache(cache, k, v, slots, ref)
    s = torch.from_numpy(slots).to(DEV)
    gpu_lib.kv4_write(cache, k.to(DEV), v.to(DEV), s)
    torch.cuda.synchronize()
    assert np.array_equal(host(cache.data)[:cache.nbytes], ref)
    ok = (slots >= 0) & (slots < cap)
    for out in (torch.float16, torch.bfloat16, torch.float32):
        rk, rv = gpu_lib.kv4_read(cache, s, out_dtype=out)
        torch.cuda.synchronize()
        for got, want in ((rk, kd), (rv, vd)):
            got = host(got).astype(np.float64)
            tol = np.abs(want) * (HALF[out] * (1 + 2.0 ** -23) + 2.0 ** -24) + TINY[out]
            assert (np.abs(got - want) <= tol)[ok].all()
            assert not got[~ok].any()


def test_kv4_strided_and_repeated(gpu_lib):
    """K and V as slices of a fused product's output, outputs likewise; the same
    slot read twice; nothing at all."""
    say("kv4 strided")
    n, heads, d = 37, 4, 64
    qkv = randn(n, 16 * d, seed=40, dtype=torch.float16).to(DEV)
    k, v = qkv[:, 8 * d:12 * d].view(n, heads, d), qkv[:, 12 * d:].view(n, heads, d)
    cache = gpu_lib.Kv4Cache(3, 64, heads, d)
    slots = torch.randperm(192, generator=gen(41))[:n].to(DEV)
    gpu_lib.kv4_write(cache, k, v, slots)
    plain = gpu_lib.Kv4Cache(3, 64, heads, d)
    gpu_lib.kv4_write(plain, k.contiguous(), v.contiguous(), slots)
    torch.cuda.synchronize()
    assert torch.equal(cache.data, plain.data)
    again = torch.cat([slots, slots[:5], slots[:1]])
    rk, rv = gpu_lib.kv4_read(cache, again)
    wide = torch.full((len(again), 2 * heads + 3, d), 7.0, dtype=torch.float16, device=DEV)
    gpu_lib.kv4_read(cache, again, k_out=wide[:, :heads], v_out=wide[:, heads + 1:2 * heads + 1])
    torch.cuda.synchronize()
    assert torch.equal(wide[:, :heads], rk) and torch.equal(wide[:, heads + 1:2 * heads + 1], rv)
    assert (wide[:, heads] == 7).all() and (wide[:, 2 * heads + 1:] == 7).all()
    assert torch.equal(rk[:5], rk[n:n + 5]) and torch.equal(rk[0], rk[-1])
    before = cache.data.clone()
    gpu_lib.kv4_write(cache, k[:0], v[:0], slots[:0])
    assert gpu_lib.kv4_read(cache, slots[:0])[0].shape == (0, heads, d)
    torch.cuda.synchronize()
    assert torch.equal(cache.data, before)


def test_kv4_extreme_values(gpu_lib):
    """Ranges past fp16, and ranges so narrow that the scale is subnormal or
    zero: bytes as the reference has them, all finite."""
    say("kv4 extremes")
    x = torch.zeros(6, 1, 64)
    x[0, 0, 0], x[0, 0, 1] = -3e38, 3e38
    x[1, 0] = torch.linspace(-1e5, 1e5, 64)
    x[2, 0] = torch.linspace(0, 3e-7, 64)
    x[3, 0] = torch.linspace(1, 1 + 1e-6, 64)
    x[4, 0] = torch.linspace(-6e4, -5e4, 64)
    x[5, 0] = -0.0
    cache = gpu_lib.Kv4Cache(1, 32, 1, 64)
    ref = np.zeros(cache.nbytes, np.uint8)
    slots = np.arange(6)
    oracle_cache(cache, x, x.flip(0), slots, ref)
    gpu_lib.kv4_write(cache, x.to(DEV), x.flip(0).to(DEV), torch.from_numpy(slots).to(DEV))
    torch.cuda.synchronize()
    assert np.array_equal(host(cache.data), ref)


# ------------------------------------------------------------- attention ---

def stored(x):
    """What the cache holds of x: values, and per value s (|c - 7.5| + 0.5) and
    23 s + |z|."""
    c, sc, z = attn_ref.quantise(host(x))
    g = c.shape[:-1] + (c.shape[-1] // 64, 64)
    s64 = np.broadcast_to(sc.astype(np.float64)[..., None], g)
    z64 = np.broadcast_to(np.abs(z.astype(np.float64))[..., None], g)
    return (attn_ref.dequantise(c, sc, z), (s64 * (np.abs(c.reshape(g) - 7.5) + 0.5)).reshape(c.shape),
            (23 * s64 + z64).reshape(c.shape))


def attn_reference(q, k, v, scale, dtype):
    """out, lse and their bounds; k and v from stored().

    A score is a sum over d of q (z + s c) taken as s (q . c) + z sum(q): D terms
    of q times a code (up to 15 s) or z, exact or one step each, added in fp32 in
    an order of their own: at most D + 8 half steps of the sum of magnitudes,
    15 s + |z| <= 3 max |k|.  The terms of the result, p s c (c <= 15) and
    p (z + mid s) (mid <= 8), are added in fp32, 32 tokens at a time and in up to
    64 shares: at most L / 32 + 64 half steps of p (23 s + |z|)."""
    d = q.shape[-1]
    kd, (vd, vround, vsum) = k[0], v
    ds = (d + 8) * 2.0 ** -24 * scale * np.abs(q).sum(-1).max() * 3 * np.abs(kd).max() if kd.size and q.size else 0.0
    vmag = 2.0 ** -11 * vround + 2.0 ** -24 * (len(kd) / 32 + 64) * vsum + 2 * ds * np.abs(vd)
    ref, lse, mag = attn_ref.attention(q, kd, vd, scale, vmag)
    return ref, (mag + np.abs(ref) * HALF[dtype] + TINY[dtype]) * (1 + 2.0 ** -8), lse, ds + 2.0 ** -20


class Batch:
    """A cache filled with NaN scales wherever no token lies, sequences on
    shuffled pages, and their exact attention."""

    def __init__(self, lib, qs, ls, hq, hkv, d, page_size, dtype, seed, cu=True, q_scale=1.0, spare=2):
        rng = np.random.default_rng(seed)
        need = [-(-length // page_size) for length in ls]
        width = max(1, max(need)) + 1
        n_pages = sum(need) + spare
        perm = rng.permutation(n_pages)
        table = np.full((len(ls), width), -7, np.int32)
        at = 0
        for i, c in enumerate(need):
            table[i, :c] = perm[at:at + c]
            at += c
        self.cache = lib.Kv4Cache(n_pages, page_size, hkv, d)
        self.cache.data.fill_(0xFF)
        self.qs, self.ls, self.hq, self.d, self.dtype, self.lib = qs, ls, hq, d, dtype, lib
        self.q = (randn(sum(qs), hq, d, seed=seed) * q_scale).to(dtype)
        self.kd, self.vd = [], []
        self.scale = d ** -0.5
        for i, length in enumerate(ls):
            k, v = make_kv(length, hkv, d, dtype, seed + 10 * i + 1) if length else (torch.zeros(0, hkv, d),) * 2
            self.kd.append(stored(k))
            self.vd.append(stored(v))
            j = np.arange(length)
            slots = table[i, j // page_size].astype(np.int64) * page_size + j % page_size
            if length:
                lib.kv4_write(self.cache, k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV))
        self.table = torch.from_numpy(table).to(DEV)
        self.lens = torch.tensor(ls, dtype=torch.int32, device=DEV)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(qs)]), dtype=torch.int32, device=DEV) if cu else None

    def run(self, **kw):
        args = dict(cu_q=self.cu, max_q=max(self.qs), max_kv=max(self.ls), want_lse=True, scale=self.scale)
        args.update(kw)
        return self.lib.kv4_attn(self.cache, self.q.to(DEV), self.table, self.lens, **args)

    def check(self, out, lse, seqs=None):
        at = 0
        for i, n in enumerate(self.qs):
            if seqs is None or i in seqs:
                q = host(self.q[at:at + n]).astype(np.float64)
                ref, tol, rl, ltol = attn_reference(q, self.kd[i], self.vd[i], self.scale, self.dtype)
                got = host(out[at:at + n]).astype(np.float64)
                err = np.abs(got - ref)
                assert (err <= tol).all(), (i, np.nanmax(err - tol), np.isnan(got).sum())
                if lse is not None:
                    gl = host(lse[at:at + n]).astype(np.float64)
                    empty = np.isneginf(rl)
                    assert np.array_equal(np.isneginf(gl), empty)
                    lerr = np.abs(gl[~empty] - rl[~empty])
                    assert (lerr <= ltol + np.abs(rl[~empty]) * 2.0 ** -22).all(), lerr.max()
            at += n


HEADS = [(4, 1, 64), (6, 2, 128), (3, 3, 64), (16, 1, 128), (40, 2, 64)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("page_size", [32, 128])
def test_attn_one_token(gpu_lib, hq, hkv, d, dtype, page_size):
    """One token per sequence; lengths of zero and one, ends inside a block and a
    page, exact block multiples, and long enough for several splits."""
    say("attn one token", hq, hkv, d, dtype, page_size)
    ls = [0, 1, 2, 31, 32, 33, 63, 65, 127, 129, 500, 1031]
    b = Batch(gpu_lib, [1] * len(ls), ls, hq, hkv, d, page_size, dtype, 300 + hq)
    b.check(*b.run())


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attn_few_tokens(gpu_lib, hq, hkv, d, dtype):
    """Several new tokens per sequence, ragged, one with none; rows before the
    cache's first token see nothing."""
    say("attn few tokens", hq, hkv, d, dtype)
    qs, ls = [5, 0, 1, 7, 3, 9, 2], [5, 40, 77, 3, 300, 64, 0]
    b = Batch(gpu_lib, qs, ls, hq, hkv, d, 64, dtype, 400 + hq)
    b.check(*b.run())


@pytest.mark.parametrize("hq,hkv,d,n,length", [(4, 1, 64, 130, 130), (8, 2, 128, 67, 300), (3, 3, 64, 257, 400),
                                               (14, 2, 128, 40, 41), (16, 1, 64, 100, 37), (2, 2, 128, 129, 1000)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attn_chunks(gpu_lib, hq, hkv, d, n, length, dtype):
    """Prompt chunks: whole prompts, later chunks, more tokens than cached."""
    say("attn chunk", hq, hkv, d, n, length, dtype)
    b = Batch(gpu_lib, [n, 3, n // 2], [length, 3, length // 3], hq, hkv, d, 32, dtype, 500 + n)
    b.check(*b.run())


def test_attn_long_and_splits(gpu_lib):
    """A long axis: the number of splits (from max_kv) changes the result by
    rounding only, results repeat bit for bit, and a workspace's content and
    size beyond need do not matter."""
    say("attn long")
    for hq, hkv, d, dtype in ((8, 2, 64, torch.float16), (4, 4, 128, torch.bfloat16)):
        b = Batch(gpu_lib, [1, 1], [9001, 20], hq, hkv, d, 64, dtype, 600 + d)
        outs = []
        for max_kv in (9001, 100, 0, 1 << 30):
            o, lse = b.run(max_kv=max_kv)
            b.check(o, lse)
            ws = gpu_lib.kv4_attn_workspace(b.cache, 2, hq, 2, 1, max_kv)
            big = torch.full((ws.numel() + 100,), 0xFF, dtype=torch.uint8, device=DEV)
            o2, lse2 = b.run(max_kv=max_kv, workspace=big)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
            outs.append(o)


def test_attn_uniform_strided_out_of_place(gpu_lib):
    """Without cu_q; q as a slice of a wider buffer in another order of axes;
    out likewise; rows behind the last sequence stay as they were."""
    say("attn strided")
    b = Batch(gpu_lib, [2] * 3, [50, 2, 130], 8, 2, 64, 32, torch.float16, 700, cu=False)
    o, lse = b.run()
    b.check(o, lse)
    wide = torch.zeros(8, 6, 3 * 64, dtype=torch.float16, device=DEV)
    qv = wide[:, :, 64:128].transpose(0, 1)  # [token][head] over a [head][token] buffer
    qv.copy_(b.q.to(DEV))
    ov = torch.full((8, 6, 128), 5.0, dtype=torch.float16, device=DEV)
    gpu_lib.kv4_attn(b.cache, qv, b.table, b.lens, max_q=2, max_kv=130, out=ov[:, :, 64:].transpose(0, 1))
    torch.cuda.synchronize()
    assert torch.equal(ov[:, :, 64:].transpose(0, 1), o) and (ov[:, :, :64] == 5).all()
    # rows outside every sequence, before and behind
    q = torch.cat([b.q[:1], b.q, b.q[:3]]).to(DEV)
    cu = torch.tensor([1, 3, 5, 7], dtype=torch.int32, device=DEV)
    for max_kv in (130, 100000):
        out = torch.full_like(q, 9.0)
        l2 = torch.full((10, 8), 9.0, device=DEV)
        gpu_lib.kv4_attn(b.cache, q, b.table, b.lens, cu_q=cu, max_q=2, max_kv=max_kv, out=out, lse=l2)
        torch.cuda.synchronize()
        b.check(out[1:7], l2[1:7])
        assert (out[[0, 7, 8, 9]] == 9).all() and (l2[[0, 7, 8, 9]] == 9).all()


def test_attn_bad_tables_and_lengths(gpu_lib):
    """Page numbers out of range hide their tokens; lengths past the table count
    to its end, negative ones as nothing; cu_q past the buffer is cut."""
    say("attn bad tables")
    b = Batch(gpu_lib, [1] * 4, [96, 96, 96, 96], 4, 2, 64, 32, torch.float16, 800)
    table = b.table[:, :3].contiguous()
    table[1, 1] = b.cache.n_pages        # the middle third is gone
    table[2, 0] = -1
    lens = torch.tensor([10 ** 9, 96, 96, -5], dtype=torch.int32, device=DEV)
    out, lse = b.lib.kv4_attn(b.cache, b.q.to(DEV), table, lens, cu_q=b.cu, max_kv=96, want_lse=True, scale=b.scale)
    torch.cuda.synchronize()
    b.check(out, lse, seqs=[0])
    for s, keep in ((1, np.r_[0:32, 64:96]), (2, np.r_[32:96])):
        q = host(b.q[s:s + 1]).astype(np.float64)
        kept = [[a[keep] for a in x] for x in (b.kd[s], b.vd[s])]
        ref, tol, _, _ = attn_reference(q, *kept, b.scale, b.dtype)
        assert (np.abs(host(out[s:s + 1]).astype(np.float64) - ref) <= tol).all()
    assert not out[3].any() and torch.isneginf(lse[3]).all()
    cu = torch.tensor([0, 1, 2, 3, 99], dtype=torch.int32, device=DEV)
    o2, _ = b.lib.kv4_attn(b.cache, b.q.to(DEV), b.table, b.lens, cu_q=cu, max_q=1, max_kv=96, scale=b.scale)
    torch.cuda.synchronize()
    b.check(o2, None)
    # one page table row for every sequence
    shared = b.table[:1].expand(4, -1)
    o3, _ = b.lib.kv4_attn(b.cache, b.q[:1].expand(4, -1, -1).to(DEV), shared, b.lens, max_kv=96, scale=b.scale)
    torch.cuda.synchronize()
    assert all(torch.equal(o3[i], o3[0]) for i in range(4))
    b.check(o3[:1], None, seqs=[0])


@pytest.mark.parametrize("q_scale", [0.0, 1e-6, 30.0])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attn_query_ranges(gpu_lib, q_scale, dtype):
    """All-zero queries (a plain mean), tiny ones, and ones so large that the
    softmax is nearly one token (the running maximum rises again and again)."""
    say("attn query range", q_scale, dtype)
    b = Batch(gpu_lib, [1, 4, 40], [700, 333, 90], 8, 2, 128, 64, dtype, 900, q_scale=q_scale)
    b.check(*b.run())


def test_attn_sink(gpu_lib):
    """One token with nearly all the weight before thousands that share the
    rest, in both orders."""
    say("attn sink")
    for where in (0, 4095):
        b = Batch(gpu_lib, [1], [4096], 4, 1, 64, 64, torch.float16, 1000)
        k = torch.zeros(4096, 1, 64)
        k[where] = 1.0
        v = randn(4096, 1, 64, seed=1001)
        b.q = torch.full((1, 4, 64), 1.4, dtype=torch.float16)
        b.kd, b.vd = [stored(k)], [stored(v)]
        j = torch.arange(4096, device=DEV)
        slots = b.table[0].long()[j // 64] * 64 + j % 64
        b.lib.kv4_write(b.cache, k.to(DEV), v.to(DEV), slots)
        b.check(*b.run())


def test_attn_nonfinite_query_stays_in_its_row(gpu_lib):
    say("attn NaN row")
    b = Batch(gpu_lib, [3, 2], [80, 40], 4, 2, 64, 32, torch.bfloat16, 1100)
    good, _ = b.run()
    b.q[1, 2, 5] = float("nan")
    b.q[3, 0, 0] = float("inf")
    bad, _ = b.run()
    torch.cuda.synchronize()
    assert torch.isnan(bad[1, 2]).all() and not torch.isfinite(bad[3, 0]).all()
    keep = torch.ones(5, 4, dtype=torch.bool)
    keep[1, 2] = keep[3, 0] = False
    assert torch.equal(bad[keep.to(DEV)], good[keep.to(DEV)])


@pytest.mark.parametrize("qs,ls,bound,hq,hkv,d", [
    ([130, 3, 64], [130, 200, 64], 200, 4, 1, 64),   # one tile a wave, a chip hardly used
    ([100, 129], [300, 290], 2100, 40, 10, 64),      # one by its rows, two by its length
    ([33], [310], 4100, 20, 5, 128),                 # little to share out: one
    ([140], [300], 4000, 176, 176, 64),              # four: long, and heads that fill the chip
    ([140], [300], 4000, 176, 176, 128),             # two at most
    ([65] * 4, [65] * 4, 65, 192, 96, 128)])         # short, but several times the chip
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attn_tiles_of_rows(gpu_lib, qs, ls, bound, hq, hkv, d, dtype):
    """Sizes on the several sides of the rule for rows per workgroup (which goes
    by the bound of the lengths)."""
    say("attn tiles of rows", qs, ls, bound, hq, hkv, d, dtype)
    b = Batch(gpu_lib, qs, ls, hq, hkv, d, 64, dtype, 1400 + d)
    b.check(*b.run(max_kv=bound))


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (16, 1, 64), (6, 2, 128), (12, 1, 128)])
@pytest.mark.parametrize("ls", [[1, 7, 40], [200, 3000], [20000]])
def test_attn_fp16_precision(gpu_lib, hq, hkv, d, ls):
    """fp16 results of up to 16 rows carry little beside their own rounding.  P is
    held in two fp16 numbers, 2^-22 of each term at most, and sums in fp32:
    (L / 32 + 64) 2^-24 of the terms' magnitudes, whose sum is at most sqrt(L)
    times what independent values leave of it.  At L = 20000 that is 141
    (2^-22 + 2^-14.5) < 0.006, but of errors as often up as down: their root over
    the L / 32 + 64 additions, 141 * 2^-24 * 26 = 0.0002, is the largest that a
    sum of random signs reaches, and as a norm it is a quarter of that or less.
    The rounding's own norm is 0.0002; so 1.25 times it holds with room, where one
    fp16 number for P gives 1.4."""
    say("attn fp16 precision", hq, hkv, d, ls)
    b = Batch(gpu_lib, [1] * len(ls), ls, hq, hkv, d, 32, torch.float16, 1300 + hq)
    out, _ = b.run()
    err = own = 0.0
    for i in range(len(ls)):
        ref = attn_reference(host(b.q[i:i + 1]).astype(np.float64), b.kd[i], b.vd[i], b.scale, b.dtype)[0]
        err += ((host(out[i:i + 1]).astype(np.float64) - ref) ** 2).sum()
        own += ((ref.astype(np.float16).astype(np.float64) - ref) ** 2).sum()
    assert err <= 1.25 ** 2 * own, (err / own) ** 0.5


def test_attn_far_pages(gpu_lib):
    """Pages whose bytes lie past 32-bit offsets."""
    say("attn far pages")
    d, hkv, page = 128, 8, 256
    per = 8 * 8 * (32 * d + 512)
    n_pages = (5 << 30) // per
    cache = gpu_lib.Kv4Cache(n_pages, page, hkv, d, data=torch.empty(5 << 30, dtype=torch.uint8, device=DEV))
    k, v = make_kv(300, hkv, d, torch.float16, 1200)
    table = torch.tensor([[n_pages - 1, n_pages // 2]], dtype=torch.int32, device=DEV)
    j = torch.arange(300, device=DEV)
    slots = table[0].long()[j // page] * page + j % page
    gpu_lib.kv4_write(cache, k.to(DEV), v.to(DEV), slots)
    rk, _ = gpu_lib.kv4_read(cache, slots, out_dtype=torch.float32)
    kd, vd = stored(k), stored(v)
    assert np.abs(host(rk) - kd[0]).max() <= np.abs(kd[0]).max() * 2.0 ** -23
    q = randn(2, 16, d, seed=1201, dtype=torch.float16)
    out, _ = gpu_lib.kv4_attn(cache, q.to(DEV), table, torch.tensor([300], dtype=torch.int32, device=DEV), max_q=2)
    ref, tol, _, _ = attn_reference(host(q).astype(np.float64), kd, vd, d ** -0.5, torch.float16)
    assert (np.abs(host(out) - ref) <= tol).all()


# ------------------------------------------------------- the run together ---

def decode_layer(lib, w, cache, x, cos, sin, pos, slots, table, lens, bufs):
    """q|k|v product, norms and rotation, cache write, attention, o product."""
    qkv, q, k, att, o, ws = bufs
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    lib.gemv_quant(*w["qkv"], x, out=qkv)
    f = qkv.view(1, hq + 2 * hkv, d)
    lib.qk_norm_rope(f[:, :hq], f[:, hq:hq + hkv], cos, sin, pos, q_weight=w["nq"], k_weight=w["nk"], q_out=q, k_out=k)
    lib.kv4_write(cache, k, f[:, hq + hkv:], slots)
    lib.kv4_attn(cache, q, table, lens, max_kv=4096, out=att, workspace=ws)
    lib.gemv_quant(*w["o"], att.view(-1), out=o)


def make_layer(lib, hq, hkv, d, width, seed):
    rows = (hq + 2 * hkv) * d
    w = {"qkv": lib.pack((randn(rows, width, seed=seed) * 0.05).to(DEV)),
         "o": lib.pack((randn(width, hq * d, seed=seed + 1) * 0.05).to(DEV)),
         "nq": (1 + 0.1 * randn(d, seed=seed + 2)).to(DEV), "nk": (1 + 0.1 * randn(d, seed=seed + 3)).to(DEV)}
    f16 = dict(dtype=torch.float16, device=DEV)
    cache = lib.Kv4Cache(64, 64, hkv, d)
    bufs = (torch.empty(rows, **f16), torch.empty(1, hq, d, **f16), torch.empty(1, hkv, d, **f16),
            torch.empty(1, hq, d, **f16), torch.empty(width, **f16), lib.kv4_attn_workspace(cache, 1, hq, 1, 1, 4096))
    return w, cache, bufs


def test_decode_layer_together(gpu_lib):
    """The operators as a decode step uses them, token after token: each step's
    attention against the reference on the queries and cached values that the
    step itself produced."""
    say("decode layer together")
    hq, hkv, d, width = 8, 2, 64, 512
    w, cache, bufs = make_layer(gpu_lib, hq, hkv, d, width, 1300)
    ang = np.arange(256)[:, None] * 500000.0 ** (-np.arange(0, d, 2) / d)
    cos, sin = (torch.from_numpy(f(ang).astype(np.float32)).to(DEV) for f in (np.cos, np.sin))
    table = torch.randperm(64, generator=gen(1301))[:4].to(torch.int32).view(1, 4).to(DEV)
    ks, vs = [], []
    for t in range(70):
        x = randn(width, seed=1400 + t, dtype=torch.bfloat16).to(DEV)
        pos = torch.tensor([t], device=DEV)
        slots = table[0, t // 64].long().view(1) * 64 + t % 64
        lens = torch.tensor([t + 1], dtype=torch.int32, device=DEV)
        decode_layer(gpu_lib, w, cache, x, cos, sin, pos, slots, table, lens, bufs)
        torch.cuda.synchronize()
        qkv, q, k, att, o, _ = bufs
        f = host(qkv).reshape(1, hq + 2 * hkv, d)
        tol = rope_tolerance(f[:, :hq], host(w["nq"]), host(cos)[[t]], host(sin)[[t]], 1e-6, d, False, torch.float16)
        ref = attn_ref.norm_rope(f[:, :hq], host(w["nq"]), host(cos)[[t]], host(sin)[[t]], 1e-6, d, False)
        assert (np.abs(host(q) - ref) <= tol).all()
        ks.append(stored(k))
        vs.append([a[None] for a in stored(torch.from_numpy(f[0, hq + hkv:].copy()))])
        if t in (0, 1, 31, 32, 63, 64, 69):
            kd, vd = ([np.concatenate(a) for a in zip(*x)] for x in (ks, vs))
            ref, tol, _, _ = attn_reference(host(q).astype(np.float64), kd, vd, d ** -0.5, torch.float16)
            assert (np.abs(host(att) - ref) <= tol).all()
            oo = gpu_lib.gemv_quant(*w["o"], att.view(-1))[1]
            assert torch.equal(oo, o)


def test_decode_layer_graph(gpu_lib):
    """The same run captured once and replayed with positions, slots and lengths
    rewritten between replays, against eager runs on a cache of its own."""
    say("decode layer graph")
    hq, hkv, d, width = 8, 2, 128, 512
    w, cache, bufs = make_layer(gpu_lib, hq, hkv, d, width, 1500)
    _, cache2, bufs2 = make_layer(gpu_lib, hq, hkv, d, width, 1500)
    cos = torch.rand(4096, d // 2, generator=gen(1501)).to(DEV)
    sin = torch.rand(4096, d // 2, generator=gen(1502)).to(DEV)
    table = torch.randperm(64, generator=gen(1503)).to(torch.int32).view(1, 64).to(DEV)
    x = torch.zeros(width, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(1, dtype=torch.int64, device=DEV)
    slots = torch.zeros(1, dtype=torch.int64, device=DEV)
    lens = torch.ones(1, dtype=torch.int32, device=DEV)

    def step(c, b):
        decode_layer(gpu_lib, w, c, x, cos, sin, pos, slots, table, lens, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, bufs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, bufs)
    for t in list(range(5)) + [63, 64, 65, 200]:
        x.copy_(randn(width, seed=1600 + t, dtype=torch.bfloat16))
        pos.fill_(t)
        slots.copy_(table[0, t // 64].long().view(1) * 64 + t % 64)
        lens.fill_(t + 1)
        graph.replay()
        torch.cuda.synchronize()
        step(cache2, bufs2)
        torch.cuda.synchronize()
        for a, b in zip(bufs[:5], bufs2[:5]):
            assert torch.equal(a, b)
        assert torch.equal(cache.data, cache2.data)


def test_two_streams_with_a_workspace_each(gpu_lib):
    """Two calls at once on streams of their own."""
    say("two streams")
    bs = [Batch(gpu_lib, [1], [5000], 8, 2, 64, 64, torch.float16, 1700 + i) for i in range(2)]
    want = [b.run() for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    got = [[], []]
    for _ in range(5):
        for i, (b, s) in enumerate(zip(bs, streams)):
            with torch.cuda.stream(s):
                got[i].append(b.run())
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_decode_pipeline_with_attention(gpu_lib):
    """The benchmark's decode pipeline with its attention run: its graph replays
    what its eager run gives (graph_time checks every output)."""
    import bench
    import synth

    say("decode pipeline with attention")
    _, probs = bench.build_layer_replicas(torch, gpu_lib, synth, synth.LLAMA32_1B_LAYER, 1, 2)
    res = bench.f4_decode_token_attention(torch, gpu_lib, probs, 1, 100, steps=3)
    assert res["layers"] == 1 and res["cached_tokens"] == 100 and res["eager_us_per_token"] > 0
    assert isinstance(res["graph_us_per_token"], float), res
