"""The operators around a layer's products on the GPU against the CPU reference
(oracle/layer_ref.py, oracle/attn_ref.py).

Tolerances, from the number formats (half a step: fp16 2^-11, bf16 2^-8, fp32
2^-24 of the value):
  norm: codes, scales and residual bit for bit.
  gate: act(g) up carries at most GATE_STEPS half steps (see gate_bound()), a
    code's quotient twice that and its own rounding, and the code half a unit.
  append: bytes and q bit for bit those of the two calls that it joins.
  attention: as tests/test_attn_gpu.py derives, over what the window leaves.
"""
import numpy as np
import pytest
import torch

from oracle import act_ref, attn_ref, layer_ref
from tests.test_attn_gpu import DEV, HALF, TINY, Batch, gen, host, make_kv, randn, say, stored

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def rounded(h, dtype):
    """fp32 numpy to a type and back"""
    return host(torch.from_numpy(np.ascontiguousarray(h)).to(dtype))


# -------------------------------------------------------------- the norm ---

def check_norm(lib, x, r, w, eps=1e-6, **outs):
    keep = None if r is None else r.clone()
    q, s, ro = lib.rms_norm_quant(x, w, residual=r, eps=eps, **outs)
    torch.cuda.synchronize()
    rq, rs, h = layer_ref.rms_norm_quant(host(x), None if r is None else host(keep), host(w), eps)
    assert np.array_equal(host(s).view(np.uint32), rs.view(np.uint32)), np.flatnonzero(host(s) != rs)
    assert np.array_equal(host(q), rq), np.argwhere(host(q) != rq)[:5]
    if r is None:
        assert ro is None
    else:
        assert ro.dtype == r.dtype and np.array_equal(host(ro), rounded(h, r.dtype))
    return q, s, ro


def norm_inputs(m, k, x_dt, r_dt, seed, pad=0):
    x = randn(m, k + pad, seed=seed).to(x_dt).to(DEV)[:, :k]
    r = None if r_dt is None else (randn(m, k, seed=seed + 1) * (1 + 20 * (randn(k, seed=seed + 2) > 2.5))).to(r_dt).to(DEV)
    return x, r, (1 + 0.3 * randn(k, seed=seed + 3)).to(DEV)


NORM_SIZES = [(1, 1), (1, 7), (3, 64), (2, 100), (1, 511), (5, 512), (1, 2048), (33, 2048), (7, 2056), (2, 4096), (3, 5001),
              (1, 8192), (2, 8200), (1, 16384), (2, 16392), (1, 32768), (1, 40001)]


@pytest.mark.parametrize("m,k", NORM_SIZES)
@pytest.mark.parametrize("x_dt,r_dt", [(torch.float16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                       (torch.float32, torch.float16), (torch.float16, None)])
def test_norm(gpu_lib, m, k, x_dt, r_dt):
    say("norm", m, k, x_dt, r_dt)
    check_norm(gpu_lib, *norm_inputs(m, k, x_dt, r_dt, 900 + k))


@pytest.mark.parametrize("m,k", [(700, 320), (3000, 64), (300, 1160), (1500, 24), (260, 2049)])
def test_norm_many_rows(gpu_lib, m, k):
    """More rows than workgroups of one launch shape take at once."""
    say("norm many rows", m, k)
    check_norm(gpu_lib, *norm_inputs(m, k, torch.bfloat16, torch.float32, 17))


@pytest.mark.parametrize("pad", [1, 3, 8, 24])
@pytest.mark.parametrize("k", [2048, 1000, 129])
def test_norm_strides(gpu_lib, pad, k):
    """x as columns of a wider matrix from an odd place on, outputs into wider ones
    whose other columns stay; the same rows from plain memory give the same."""
    say("norm strides", pad, k)
    m = 6
    wide = randn(m, k + 2 * pad, seed=3).half().to(DEV)
    x, r = wide[:, pad:pad + k], randn(m, k + pad, seed=4).to(DEV)[:, :k]
    w = (1 + 0.1 * randn(k, seed=5)).to(DEV)
    q_wide = torch.full((m, k + 2 * pad), 77, dtype=torch.int8, device=DEV)
    ro_wide = torch.full((m, k + pad), 55.0, device=DEV)
    q, s, ro = check_norm(gpu_lib, x, r, w, q_out=q_wide[:, pad:pad + k], residual_out=ro_wide[:, :k])
    q2, s2, ro2 = gpu_lib.rms_norm_quant(x.contiguous(), w, residual=r.contiguous())
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(ro, ro2)
    assert (q_wide[:, :pad] == 77).all() and (q_wide[:, pad + k:] == 77).all() and (ro_wide[:, k:] == 55).all()


@pytest.mark.parametrize("m,k", [(1, 2048), (40, 2048), (3, 1001), (2, 40000)])
@pytest.mark.parametrize("r_dt", [torch.float32, torch.bfloat16])
def test_norm_residual_in_place(gpu_lib, m, k, r_dt):
    say("norm in place", m, k, r_dt)
    x, r, w = norm_inputs(m, k, torch.float16, r_dt, 31)
    want = gpu_lib.rms_norm_quant(x, w, residual=r)
    mine = r.clone()
    got = check_norm(gpu_lib, x, mine, w, residual_out=mine)
    assert got[2].data_ptr() == mine.data_ptr()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("k", [512, 1001, 40000])
def test_norm_extreme_rows(gpu_lib, k):
    """Zeros (scale 1), sizes whose squares pass fp32, subnormal ones, a residual
    that cancels x, and a row with a NaN or an infinity between sound ones."""
    say("norm extremes", k)
    x = randn(9, k, seed=6)
    x[0] = 0
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = 1e-42
    x[4, :] = 0
    x[4, k // 2] = -5.0
    r = torch.zeros(9, k)
    r[5] = -x[5]
    x[6, k - 1] = float("nan")
    x[7, 0] = float("inf")
    w = (1 + 0.3 * randn(k, seed=7)).to(DEV)
    for eps in (0.0, 1e-5):
        q, s, ro = gpu_lib.rms_norm_quant(x.to(DEV), w, residual=r.to(DEV), eps=eps)
        torch.cuda.synchronize()
        ok = [1, 2, 4, 8] if eps == 0 else [0, 1, 2, 3, 4, 5, 8]  # (0 / 0 without eps; 1e-42 has no square in fp64's reach)
        with np.errstate(all="ignore"):
            rq, rs, h = layer_ref.rms_norm_quant(x[ok].numpy(), r[ok].numpy(), host(w), eps)
        assert np.array_equal(host(q)[ok], rq) and np.array_equal(host(s)[ok], rs)
        assert np.array_equal(host(ro)[ok], h)


def test_norm_feeds_the_products(gpu_lib):
    """Codes and scales are what gemm takes: the product of both is the oracle's
    on the reference's codes."""
    from oracle import sherry_ref

    say("norm into gemm")
    n, k, m = 64, 512, 5
    words = torch.randint(-2 ** 31, 2 ** 31 - 1, (n * k * 5 // 128,), generator=gen(1), dtype=torch.int64).to(torch.int32)
    scales = torch.rand(n, generator=gen(2)) * 0.1
    x, r, w = norm_inputs(m, k, torch.float16, torch.float32, 50)
    q, s, _ = check_norm(gpu_lib, x, r, w)
    acc, y = gpu_lib.gemm(words.to(DEV), scales.to(DEV), q, s, torch.float32, want_acc=True)
    racc, ry = sherry_ref.gemm_i8(words.numpy().view(np.uint32), scales.numpy(), n, k, host(q), host(s), np.float32)
    assert np.array_equal(host(acc), racc) and np.array_equal(host(y), ry)


# -------------------------------------------------------- the gated rows ---

def gate_bound(g, act):
    """Relative error of act(g) up in half steps of fp32: the exponential (a step
    of its own and half a step of its argument z times log2 e, both below the next
    power of two of |z|), its sum with 1, the quotient (two steps where it is a
    reciprocal's), the product: 2 + 1 + 4 + 1.  z itself is g, or off by 4 half
    steps of itself (three products and a sum), which the exponential multiplies by
    |z|; where exp(-z) is nothing beside 1 none of that shows, so |z| counts where
    z < 0 or by its share exp(-z)."""
    g = np.asarray(g, np.float64)
    z = g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    share = 1 / (1 + np.exp(np.minimum(z, 700.0)))  # exp(-z) / (1 + exp(-z))
    return 8 + share * np.abs(z) * (2 if act == "silu" else 6)


def check_gated(lib, g, u, act, **outs):
    q, s = lib.gated_quant(g, u, activation=act, **outs)
    torch.cuda.synchronize()
    g64, u64 = host(g).astype(np.float64), host(u).astype(np.float64)
    y = layer_ref.gated(g64, u64, act)
    bound = gate_bound(g64, act) * 2.0 ** -24 * np.abs(y) + 2.0 ** -119 * np.abs(u64)  # (exp past fp32: 0)
    top = np.abs(y).max(-1)
    top_off = np.array([b[np.abs(v) >= t * (1 - 1e-4)].max() for b, v, t in zip(bound, y, top)])
    want_s = np.where(top == 0, 1.0, top / 127)
    got_s = host(s).astype(np.float64)
    s_off = top_off / 127 + 2.0 ** -24 * want_s + 2.0 ** -149
    assert (np.abs(got_s - want_s) <= s_off).all(), (got_s, want_s)
    t = y / want_s[:, None]
    off = bound / want_s[:, None] + np.abs(t) * ((s_off / want_s)[:, None] + 2.0 ** -24)
    c = host(q).astype(np.float64)
    assert (np.abs(c - t) <= 0.5 + off * 1.001).all(), np.max(np.abs(c - t) - 0.5 - off)
    assert np.abs(c).max(-1).min() >= 127 or (top == 0).any()
    return q, s


@pytest.mark.parametrize("m,k", NORM_SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated(gpu_lib, m, k, dtype, act):
    say("gated", m, k, dtype, act)
    gu = (randn(m, 2 * k, seed=60 + k) * 2).to(dtype).to(DEV)
    check_gated(gpu_lib, gu[:, :k], gu[:, k:], act)


@pytest.mark.parametrize("m,k", [(700, 320), (3000, 64), (300, 1160), (1500, 24), (260, 2049)])
def test_gated_many_rows(gpu_lib, m, k):
    say("gated many rows", m, k)
    check_gated(gpu_lib, randn(m, k, seed=61).half().to(DEV), randn(m, k, seed=62).half().to(DEV), "silu")


@pytest.mark.parametrize("k", [1024, 999])
@pytest.mark.parametrize("pad", [1, 8])
def test_gated_strides(gpu_lib, k, pad):
    """Halves of a wider matrix in either order, codes into a wider one."""
    say("gated strides", k, pad)
    m = 5
    wide = randn(m, 2 * k + 3 * pad, seed=63).to(torch.bfloat16).to(DEV)
    up, gate = wide[:, pad:pad + k], wide[:, 2 * pad + k:2 * pad + 2 * k]
    q_wide = torch.full((m, k + 2 * pad), 77, dtype=torch.int8, device=DEV)
    q, s = check_gated(gpu_lib, gate, up, "silu", q_out=q_wide[:, pad:pad + k])
    q2, s2 = gpu_lib.gated_quant(gate.contiguous(), up.contiguous())
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert (q_wide[:, :pad] == 77).all() and (q_wide[:, pad + k:] == 77).all()


@pytest.mark.parametrize("k", [512, 1001, 40000])
def test_gated_extreme_rows(gpu_lib, k):
    """Large gates of both signs, zeros on either side, tiny values; a row with a
    NaN between sound ones."""
    say("gated extremes", k)
    g, u = randn(8, k, seed=64), randn(8, k, seed=65)
    g[0] = 0
    u[1] = 0
    g[2] *= 60
    g[3] = torch.linspace(-200, 200, k)
    g[4] *= 1e-20
    u[5] *= 1e30
    g[6, 3] = float("nan")
    for act in ("silu", "gelu_tanh"):
        q, s = gpu_lib.gated_quant(g.to(DEV), u.to(DEV), activation=act)
        torch.cuda.synchronize()
        ok = [i for i in range(8) if i != 6]
        q2, s2 = check_gated(gpu_lib, g[ok].to(DEV), u[ok].to(DEV), act)
        assert torch.equal(q[ok], q2) and torch.equal(s[ok], s2)
        assert s[0] == 1 and s[1] == 1 and not q[:2].any()


# ------------------------------------------------------------ the append ---

def append_inputs(n, hq, hkv, d, rot, x_dt, norm, seed, maxpos=400):
    qkv = randn(n, (hq + 2 * hkv) * d, seed=seed).to(x_dt).to(DEV).view(n, hq + 2 * hkv, d)
    ang = randn(maxpos, rot // 2, seed=seed + 1) * 3
    w = [(1 + 0.3 * randn(d, seed=seed + 2 + i)).to(DEV) if norm else None for i in range(2)]
    return (qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], ang.cos().to(DEV), ang.sin().to(DEV),
            torch.randint(0, maxpos, (n,), generator=gen(seed + 5)).to(DEV), w)


def two_calls(lib, cache, q, k, v, cos, sin, pos, slots, w, inter, out_dtype, eps=1e-6):
    """qk_norm_rope with an fp32 k, then kv4_write: the cache of the one call."""
    rq, _ = lib.qk_norm_rope(q, None, cos, sin, pos, q_weight=w[0], eps=eps, interleaved=inter, out_dtype=out_dtype)
    _, rk = lib.qk_norm_rope(q, k, cos, sin, pos, q_weight=w[0], k_weight=w[1], eps=eps, interleaved=inter,
                             out_dtype=torch.float32)
    lib.kv4_write(cache, rk, v.float(), slots)
    return rq


HOW = {
    "one": lambda n, cap, r: r.permutation(cap)[:n],
    "run": lambda n, cap, r: np.arange(n) + 5,
    "aligned run": lambda n, cap, r: np.arange(n) + 32,
    "skips": lambda n, cap, r: np.where(r.random(n) < 0.3, r.choice([-1, cap, cap + 10 ** 12, -2 ** 62], n),
                                        r.permutation(cap)[:n]),
}


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32), (128, 96)])
@pytest.mark.parametrize("n,hq,hkv,page_size,how", [(1, 4, 1, 32, "one"), (133, 6, 3, 64, "run"), (130, 2, 2, 256, "aligned run"),
                                                    (100, 7, 1, 64, "skips"), (45, 5, 5, 32, "one")])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("x_dt,out", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16),
                                      (torch.float32, torch.float16), (torch.float16, torch.float32)])
def test_append(gpu_lib, d, rot, n, hq, hkv, page_size, how, inter, x_dt, out):
    """q and every byte of the cache, those of other tokens among them."""
    say("append", d, rot, n, hq, hkv, page_size, how, inter, x_dt, out)
    norm = n != 45
    q, k, v, cos, sin, pos, w = append_inputs(n, hq, hkv, d, rot, x_dt, norm, 70 + d + n)
    n_pages = 512 // page_size
    slots = torch.from_numpy(HOW[how](n, 512, np.random.default_rng(n)).astype(np.int64)).to(DEV)
    caches = [gpu_lib.Kv4Cache(n_pages, page_size, hkv, d) for _ in range(2)]
    for c in caches:
        c.data.fill_(0xA5)
    got = gpu_lib.kv4_append(caches[0], q, k, v, cos, sin, pos, slots, q_weight=w[0], k_weight=w[1], interleaved=inter,
                             out_dtype=out)
    want = two_calls(gpu_lib, caches[1], q, k, v, cos, sin, pos, slots, w, inter, out)
    torch.cuda.synchronize()
    assert got.dtype == out and torch.equal(got, want)
    assert torch.equal(caches[0].data, caches[1].data)


@pytest.mark.parametrize("d", [64, 128])
def test_append_against_the_reference(gpu_lib, d):
    """Without the library's own calls: q and what the cache reads back as against
    64 bits.  A stored key is off from the reference's values by half a quantiser
    step, the roundings of its scale and zero point (half a step of 15 s + |z|),
    and the rotation's own error."""
    from tests.test_attn_gpu import rope_tolerance

    say("append reference", d)
    n, hq, hkv = 70, 4, 2
    q, k, v, cos, sin, pos, w = append_inputs(n, hq, hkv, d, d, torch.float16, True, 90 + d)
    cache = gpu_lib.Kv4Cache(4, 32, hkv, d)
    slots = torch.randperm(128, generator=gen(3))[:n].to(DEV)
    got = gpu_lib.kv4_append(cache, q, k, v, cos, sin, pos, slots, q_weight=w[0], k_weight=w[1])
    rk, rv = gpu_lib.kv4_read(cache, slots, out_dtype=torch.float32)
    torch.cuda.synchronize()
    p = host(pos)
    c, s = host(cos)[p], host(sin)[p]
    ref = attn_ref.norm_rope(host(q), host(w[0]), c, s, 1e-6, d, False)
    tol = rope_tolerance(host(q), host(w[0]), c, s, 1e-6, d, False, torch.float16)
    assert (np.abs(host(got) - ref) <= tol).all()
    kref = attn_ref.norm_rope(host(k), host(w[1]), c, s, 1e-6, d, False)
    ktol = rope_tolerance(host(k), host(w[1]), c, s, 1e-6, d, False, torch.float32)
    g = kref.reshape(n, hkv, d // 64, 64)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    step = (hi - lo) / 15
    half = np.broadcast_to(0.5 * step * (1 + 2.0 ** -10) + 2.0 ** -11 * (15 * step + np.abs(lo)) + 2.0 ** -24 * 30, g.shape)
    assert (np.abs(host(rk) - kref) <= half.reshape(kref.shape) + 4 * ktol).all()
    vc = attn_ref.dequantise(*attn_ref.quantise(host(v)))
    assert (np.abs(host(rv) - vc) <= np.abs(vc) * 2.0 ** -23).all()


def test_append_without_q_strided_and_in_place(gpu_lib):
    say("append forms")
    n, hq, hkv, d = 37, 4, 2, 64
    q, k, v, cos, sin, pos, w = append_inputs(n, hq, hkv, d, d, torch.float16, True, 95)
    slots = torch.randperm(192, generator=gen(41))[:n].to(DEV)
    caches = [gpu_lib.Kv4Cache(3, 64, hkv, d) for _ in range(3)]
    want = gpu_lib.kv4_append(caches[0], q.contiguous(), k.contiguous(), v.contiguous(), cos, sin, pos, slots,
                              q_weight=w[0], k_weight=w[1])
    assert gpu_lib.kv4_append(caches[1], None, k, v, cos, sin, pos, slots, k_weight=w[1]) is None
    turned = torch.empty(hq + 2 * hkv, n, d, dtype=torch.float16, device=DEV)  # [head][token]
    turned.copy_(torch.cat([q, k, v], 1).transpose(0, 1))
    qi, ki, vi = (t.transpose(0, 1) for t in turned.split([hq, hkv, hkv]))
    got = gpu_lib.kv4_append(caches[2], qi, ki, vi, cos, sin, pos, slots, q_weight=w[0], k_weight=w[1], q_out=qi)
    torch.cuda.synchronize()
    assert got.data_ptr() == qi.data_ptr() and torch.equal(got, want)
    assert torch.equal(turned[hq:], torch.cat([k, v], 1).transpose(0, 1))
    for c in caches[1:]:
        assert torch.equal(c.data, caches[0].data)
    e = gpu_lib.kv4_append(caches[0], q[:0], k[:0], v[:0], cos, sin, pos[:0], slots[:0])
    assert e.shape == (0, hq, d)


def test_append_positions_out_of_range(gpu_lib):
    """Such a token is not written, alone or inside a whole block; its q is NaN."""
    say("append bad positions")
    n, hq, hkv, d = 96, 2, 1, 64
    q, k, v, cos, sin, pos, w = append_inputs(n, hq, hkv, d, 32, torch.float16, False, 97)
    bad = torch.tensor([3, 40, 41, 95], device=DEV)
    wrong = pos.clone()
    wrong[bad] = torch.tensor([-1, 400, 2 ** 40, -2 ** 50], device=DEV)
    slots = torch.arange(n, device=DEV)
    caches = [gpu_lib.Kv4Cache(4, 32, hkv, d) for _ in range(2)]
    for c in caches:
        c.data.fill_(0xA5)
    got = gpu_lib.kv4_append(caches[0], q, k, v, cos, sin, wrong, slots)
    off = slots.clone()
    off[bad] = -1
    want = gpu_lib.kv4_append(caches[1], q, k, v, cos, sin, pos, off)
    torch.cuda.synchronize()
    assert torch.equal(caches[0].data, caches[1].data)
    good = torch.ones(n, dtype=torch.bool, device=DEV)
    good[bad] = False
    assert torch.equal(got[good], want[good])
    assert torch.isnan(got[bad][..., :32]).all() and torch.equal(got[bad][..., 32:], q[bad][..., 32:])


# ------------------------------------------------ attention with a window ---

class WindowBatch(Batch):
    """A Batch of which only what some row sees is there: other tokens' bytes are
    NaN scales, other pages' numbers out of range or those of another page."""

    def __init__(self, lib, qs, ls, hq, hkv, d, page_size, dtype, seed, window, sinks, cu=True, q_scale=1.0):
        super().__init__(lib, qs, ls, hq, hkv, d, page_size, dtype, seed, cu=cu, q_scale=q_scale)
        self.window, self.sinks = window, sinks
        table = host(self.table).copy()
        fresh = torch.full_like(self.cache.data, 0xFF)
        old, self.cache.data = self.cache.data, fresh
        keep = self.cache
        self.cache = lib.Kv4Cache(keep.n_pages, page_size, hkv, d, data=fresh)
        from_ = lib.Kv4Cache(keep.n_pages, page_size, hkv, d, data=old)
        assert from_.n_pages == keep.n_pages
        rng = np.random.default_rng(seed + 1)
        for i, (n, length) in enumerate(zip(qs, ls)):
            seen = layer_ref.visible(n, length, window, sinks).any(0) if n else np.zeros(length, bool)
            j = np.flatnonzero(seen)
            if j.size:
                k, v = make_kv(length, hkv, d, dtype, seed + 10 * i + 1)
                slots = table[i, j // page_size].astype(np.int64) * page_size + j % page_size
                lib.kv4_write(self.cache, k[j].to(DEV), v[j].to(DEV), torch.from_numpy(slots).to(DEV))
            for page in range(-(-length // page_size)):
                if not seen[page * page_size:(page + 1) * page_size].any():
                    table[i, page] = rng.choice([-1, 10 ** 9, keep.n_pages - 1])
        self.table = torch.from_numpy(table).to(DEV)

    def run(self, **kw):
        return super().run(**{**dict(window=self.window, sinks=self.sinks), **kw})

    def check(self, out, lse, seqs=None):
        at = 0
        for i, n in enumerate(self.qs):
            if seqs is None or i in seqs:
                q = host(self.q[at:at + n]).astype(np.float64)
                ref, tol, rl, ltol = window_reference(q, self.kd[i], self.vd[i], self.scale, self.dtype, self.window, self.sinks)
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


def window_reference(q, k, v, scale, dtype, window, sinks):
    """attn_reference() of tests/test_attn_gpu.py over what the window leaves (its
    bounds grow with the tokens walked, fewer here)."""
    d = q.shape[-1]
    kd, (vd, vround, vsum) = k[0], v
    ds = (d + 8) * 2.0 ** -24 * scale * np.abs(q).sum(-1).max() * 3 * np.abs(kd).max() if kd.size and q.size else 0.0
    vmag = 2.0 ** -11 * vround + 2.0 ** -24 * (min(len(kd), window + sinks + 64) / 32 + 64) * vsum + 2 * ds * np.abs(vd)
    ref, lse, mag = layer_ref.window_attention(q, kd, vd, scale, window, sinks, vmag)
    return ref, (mag + np.abs(ref) * HALF[dtype] + TINY[dtype]) * (1 + 2.0 ** -8), lse, ds + 2.0 ** -20


W_HEADS = [(4, 1, 64), (6, 2, 128), (16, 1, 128), (40, 2, 64)]
WINDOWS = [(1, 0), (1, 1), (5, 4), (32, 32), (33, 0), (64, 31), (100, 33), (128, 70), (500, 4), (4000, 0), (40, 5000)]


@pytest.mark.parametrize("hq,hkv,d", W_HEADS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_window_one_token(gpu_lib, hq, hkv, d, window, sinks, dtype):
    """One token a sequence; lengths around the window's and the sinks' ends."""
    say("window one token", hq, hkv, d, window, sinks, dtype)
    ls = [0, 1, 2, 31, 33, 64, 65, 127, 129, 160, 500, 1031]
    b = WindowBatch(gpu_lib, [1] * len(ls), ls, hq, hkv, d, 64, dtype, 300 + hq, window, sinks)
    b.check(*b.run())


@pytest.mark.parametrize("hq,hkv,d", W_HEADS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window_few_tokens(gpu_lib, hq, hkv, d, window, sinks):
    """Several new tokens a sequence, ragged, one with none; rows before the first
    cached token see nothing."""
    say("window few tokens", hq, hkv, d, window, sinks)
    qs, ls = [5, 0, 1, 7, 3, 9, 2, 4], [5, 40, 77, 3, 300, 64, 0, 777]
    b = WindowBatch(gpu_lib, qs, ls, hq, hkv, d, 32, torch.float16, 400 + hq, window, sinks)
    b.check(*b.run())


@pytest.mark.parametrize("hq,hkv,d,n,length", [(4, 1, 64, 130, 130), (8, 2, 128, 67, 300), (3, 3, 64, 257, 400),
                                               (14, 2, 128, 40, 41), (16, 1, 64, 100, 37), (2, 2, 128, 129, 1000)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 40), (32, 4), (65, 0), (150, 33), (900, 1)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_window_chunks(gpu_lib, hq, hkv, d, n, length, window, sinks, dtype):
    """Prompt chunks: whole prompts, later chunks, more tokens than cached."""
    say("window chunk", hq, hkv, d, n, length, window, sinks, dtype)
    b = WindowBatch(gpu_lib, [n, 3, n // 2], [length, 3, length // 3], hq, hkv, d, 32, dtype, 500 + n, window, sinks)
    b.check(*b.run())


@pytest.mark.parametrize("hq,hkv,d,qs,ls", [(32, 8, 64, [600], [900]), (32, 8, 64, [1100], [1100]), (8, 2, 128, [1, 1], [9001, 20]),
                                            (8, 2, 64, [20], [5000]), (64, 4, 64, [260, 9], [2000, 500])])
@pytest.mark.parametrize("window,sinks", [(300, 20), (2500, 4)])
def test_window_splits(gpu_lib, hq, hkv, d, qs, ls, window, sinks):
    """Sizes that take larger tiles and splits; other max_kv change the splits, and
    the result by rounding only; results repeat bit for bit."""
    say("window splits", hq, hkv, d, qs, ls, window, sinks)
    b = WindowBatch(gpu_lib, qs, ls, hq, hkv, d, 64, torch.float16, 600 + d, window, sinks)
    for max_kv in (max(ls), 100, 1 << 30):
        o, lse = b.run(max_kv=max_kv)
        b.check(o, lse)
        ws = gpu_lib.kv4_attn_workspace(b.cache, sum(qs), hq, len(qs), max(qs), max_kv, window=window, sinks=sinks)
        big = torch.full((ws.numel() + 100,), 0xFF, dtype=torch.uint8, device=DEV)
        o2, lse2 = b.run(max_kv=max_kv, workspace=big)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_window_of_everything(gpu_lib):
    """A window of all that the table holds is the call without one, bit for bit;
    one that merely no row reaches gives the same up to rounding."""
    say("window of everything")
    for qs, ls in (([1] * 3, [50, 1, 700]), ([70, 3], [300, 9])):
        b = Batch(gpu_lib, qs, ls, 8, 2, 64, 32, torch.float16, 77)
        o, lse = b.run()
        cap = b.table.shape[1] * 32
        for window in (cap, cap + 1, 2 ** 40):
            o2, lse2 = b.run(window=window, sinks=3)
            torch.cuda.synchronize()
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
        b.check(*b.run(window=max(ls)))


def test_window_rows_behind_and_strides(gpu_lib):
    """q and out in other orders; rows of no sequence stay as they were; bad pages
    inside the window hide their tokens."""
    say("window rows behind")
    b = WindowBatch(gpu_lib, [2] * 3, [50, 2, 130], 8, 2, 64, 32, torch.float16, 700, 40, 3)
    o, lse = b.run()
    b.check(o, lse)
    q = torch.cat([b.q[:1], b.q, b.q[:3]]).to(DEV)
    cu = torch.tensor([1, 3, 5, 7], dtype=torch.int32, device=DEV)
    wide = torch.full((8, 10, 128), 9.0, dtype=torch.float16, device=DEV)
    l2 = torch.full((10, 8), 9.0, device=DEV)
    gpu_lib.kv4_attn(b.cache, q, b.table, b.lens, cu_q=cu, max_q=2, max_kv=130, out=wide[:, :, 64:].transpose(0, 1), lse=l2,
                     window=40, sinks=3)
    torch.cuda.synchronize()
    out = wide[:, :, 64:].transpose(0, 1)
    assert torch.equal(out[1:7], o) and torch.equal(l2[1:7], lse)
    assert (out[[0, 7, 8, 9]] == 9).all() and (l2[[0, 7, 8, 9]] == 9).all() and (wide[:, :, :64] == 9).all()
    table = b.table.clone()
    table[2] = -1  # nothing of the third sequence is there
    o2, lse2 = gpu_lib.kv4_attn(b.cache, b.q.to(DEV), table, b.lens, cu_q=b.cu, max_q=2, want_lse=True, window=40, sinks=3)
    torch.cuda.synchronize()
    assert torch.equal(o2[:4], o[:4]) and not o2[4:].any() and torch.isneginf(lse2[4:]).all()


# -------------------------------------------------------------- together ---

def test_a_layer_together(gpu_lib):
    """A decoder layer as it runs: a prompt chunk, then tokens one by one through
    norm, q|k|v, append, windowed attention, o, norm, gate|up, gate, down; decode
    steps captured in one graph and replayed, each against the same calls made
    eagerly, and the last hidden state against the layer in 64 bits on the codes
    that the GPU made."""
    say("layer together")
    hid, hq, hkv, d, ffn, page, window, sinks, chunk, steps = 512, 8, 2, 64, 1024, 32, 48, 4, 70, 5
    total = chunk + steps
    mats = {}
    for i, (name, n, k) in enumerate((("qkv", (hq + 2 * hkv) * d, hid), ("o", hid, hq * d), ("gu", 2 * ffn, hid), ("down", hid, ffn))):
        mats[name] = gpu_lib.pack((randn(n, k, seed=i) * k ** -0.5).to(DEV))
    w1, w2 = ((1 + 0.1 * randn(hid, seed=10 + i)).to(DEV) for i in range(2))
    ang = torch.arange(total)[:, None] * 10000.0 ** (-torch.arange(0, d, 2) / d)
    cos, sin = ang.cos().to(DEV), ang.sin().to(DEV)
    pages = -(-total // page)
    table = torch.randperm(pages, generator=gen(4)).to(torch.int32).view(1, pages).to(DEV)
    place = torch.arange(total, device=DEV)
    every = table[0].long()[place // page] * page + place % page
    x_in = (randn(total, hid, seed=20) * 2).to(DEV)

    def product(name, q, s):
        return gpu_lib.gemm(*mats[name], q, s)[1] if q.shape[0] > 1 else gpu_lib.gemv(*mats[name], q[0], s)[1][None]

    def layer(cache, h, pos, slots, lens):
        n = h.shape[0]
        zero = torch.zeros(n, hid, dtype=torch.float16, device=DEV)
        q, s, h1 = gpu_lib.rms_norm_quant(zero, w1, residual=h)
        qkv = product("qkv", q, s).view(n, hq + 2 * hkv, d)
        rq = gpu_lib.kv4_append(cache, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], cos, sin, pos, slots)
        att, _ = gpu_lib.kv4_attn(cache, rq, table, lens, max_q=n, max_kv=total, window=window, sinks=sinks)
        o = product("o", *gpu_lib.act_quant(att.view(n, hq * d)))
        q, s, h2 = gpu_lib.rms_norm_quant(o, w2, residual=h1)
        gu = product("gu", q, s)
        down = product("down", *gpu_lib.gated_quant(gu[:, :ffn], gu[:, ffn:]))
        return h2 + down.float(), (rq, att, o, gu, down)

    caches = [gpu_lib.Kv4Cache(pages, page, hkv, d) for _ in range(2)]
    lens = torch.tensor([chunk], dtype=torch.int32, device=DEV)
    outs = [layer(c, x_in[:chunk], place[:chunk], every[:chunk], lens)[0] for c in caches]
    torch.cuda.synchronize()
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all() and torch.equal(caches[0].data, caches[1].data)
    # one token at a time: static inputs that the graph reads
    h, pos, slot, ln = x_in[:1].clone(), place[:1].clone(), every[:1].clone(), lens.clone()
    blank = caches[1].data.clone()
    pos.fill_(chunk), slot.copy_(every[chunk:chunk + 1]), ln.fill_(chunk + 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(caches[1], h, pos, slot, ln)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, parts = layer(caches[1], h, pos, slot, ln)
    caches[1].data.copy_(blank)
    for t in range(chunk, total):
        want, want_parts = layer(caches[0], x_in[t:t + 1], place[t:t + 1], every[t:t + 1],
                                 torch.tensor([t + 1], dtype=torch.int32, device=DEV))
        h.copy_(x_in[t:t + 1]), pos.fill_(t), slot.copy_(every[t:t + 1]), ln.fill_(t + 1)
        for again in range(2):  # (a token written twice is the same token)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(parts, want_parts)), (t, again)
            assert torch.equal(caches[0].data, caches[1].data)
    # the last token's attention and feed-forward from what the GPU holds, in 64 bits
    rq, att, o, gu, down = (host(p).astype(np.float64) for p in want_parts)
    k, v = (host(a).astype(np.float64) for a in gpu_lib.kv4_read(caches[0], every, out_dtype=torch.float32))
    ref, _, mag = layer_ref.window_attention(rq, k, v, d ** -0.5, window, sinks)
    assert np.abs(att - ref).max() <= (2.0 ** -10 * mag + 2.0 ** -11 * np.abs(ref)).max()
    q, s = act_ref.quantize(layer_ref.gated(gu[:, :ffn], gu[:, ffn:], "silu").astype(np.float32))
    t = host(gpu_lib.decode(mats["down"][0], hid, ffn)).astype(np.float64)
    want = (q.astype(np.float64) @ t.T) * host(mats["down"][1]).astype(np.float64) * s[:, None]
    # a code or two may round the other way: one unit of one row's weight each
    assert np.abs(down - want).max() <= 2.0 ** -11 * np.abs(want).max() + 2.5 * s[0] * host(mats["down"][1]).max()


# ------------------------------------------------ sizes that choose variants ---

@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (128, 128, False), (64, 32, True), (128, 64, False)])
@pytest.mark.parametrize("n,hq,hkv,at", [(300, 6, 3, 0), (777, 5, 2, 13), (1500, 40, 8, 32), (2100, 33, 3, 7), (600, 0, 2, 5),
                                          (1200, 0, 2, 5), (1025, 4, 1, 0), (1024, 4, 1, 3)])
def test_append_many(gpu_lib, d, rot, inter, n, hq, hkv, at):
    """Tiles cut where blocks begin, two heads a lane (an odd head left over), k and v
    first or spread over the launch, no q; some slots and positions out of range."""
    say("append many", d, rot, inter, n, hq, hkv, at)
    q, k, v, cos, sin, pos, w = append_inputs(n, max(hq, 1), hkv, d, rot, torch.bfloat16, True, 110 + d + n)
    slots = (torch.arange(n) + at).to(DEV)
    slots[n // 2] = -3
    pages = (n + at) // 64 + 1
    caches = [gpu_lib.Kv4Cache(pages, 64, hkv, d) for _ in range(2)]
    for c in caches:
        c.data.fill_(0xA5)
    wrong = pos.clone()
    wrong[n // 3] = -1
    got = gpu_lib.kv4_append(caches[0], q if hq else None, k, v, cos, sin, wrong, slots, q_weight=w[0] if hq else None,
                             k_weight=w[1], interleaved=inter)
    off = slots.clone()
    off[n // 3] = -1
    want = two_calls(gpu_lib, caches[1], q, k, v, cos, sin, wrong, off, w, inter, torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(caches[0].data, caches[1].data)
    if hq:
        ok = torch.ones(n, dtype=torch.bool, device=DEV)
        ok[n // 3] = False
        assert torch.equal(got[ok], want[ok]) and torch.isnan(got[n // 3, :, :rot]).all()


@pytest.mark.parametrize("hq,hkv,d,qs,ls", [(32, 8, 64, [1100], [1500]), (64, 4, 64, [260, 9], [2000, 500]),
                                            (48, 8, 64, [17] * 9, [400] * 9), (24, 8, 128, [300, 7], [900, 2000]),
                                            (8, 8, 64, [2100], [2100]), (20, 1, 128, [13] * 3, [33, 700, 8])])
@pytest.mark.parametrize("window,sinks", [(100, 0), (700, 65)])
def test_window_many_rows_bf16(gpu_lib, hq, hkv, d, qs, ls, window, sinks):
    say("window many rows", hq, hkv, d, qs, ls, window, sinks)
    b = WindowBatch(gpu_lib, qs, ls, hq, hkv, d, 128, torch.bfloat16, 610 + d, window, sinks, q_scale=2.0)
    b.check(*b.run())


def test_window_max_q_cuts_a_sequence(gpu_lib):
    """Of a longer sequence only the first max_q rows are computed; the others stay."""
    say("window max_q")
    for dims in ((8, 2, 64, [40, 3], [300, 90], 9), (16, 2, 128, [200, 60], [500, 61], 50), (64, 4, 64, [300, 9], [900, 30], 270)):
        hq, hkv, d, qs, ls, max_q = dims
        b = WindowBatch(gpu_lib, qs, ls, hq, hkv, d, 32, torch.float16, 650, 77, 5)
        full, lse = b.run()
        b.check(full, lse)
        out, l2 = torch.full_like(full, 3.0), torch.full_like(lse, 3.0)
        b.run(max_q=max_q, out=out, lse=l2)
        torch.cuda.synchronize()
        at = 0
        for n in qs:
            done = min(n, max_q)
            err = (out[at:at + done].float() - full[at:at + done].float()).abs().max()
            assert err <= 2.0 ** -9 * full.float().abs().max() and (out[at + done:at + n] == 3).all()
            assert (l2[at + done:at + n] == 3).all()
            at += n


def test_window_spoiled_rows_and_huge_scores(gpu_lib):
    """A row with a NaN spoils itself alone, and queries of 2^40 in size keep finite
    rows: every other row stays within its bound.  (Not bit for bit: the maximum is
    raised for the sixteen rows of a tile together, when one of them needs it, and
    that rescales and rounds their sums anew.)"""
    say("window spoiled rows")
    for qs, ls in (([3] * 4, [200, 7, 90, 3]), ([70], [200])):
        b = WindowBatch(gpu_lib, qs, ls, 8, 2, 64, 32, torch.bfloat16, 660, 50, 4)
        o, lse = b.run()
        b.check(o, lse)
        sound = b.q.clone()
        b.q[1, 3, 5] = float("nan")
        b.q[2, 0] *= 2.0 ** 40
        o2, lse2 = b.run()
        torch.cuda.synchronize()
        assert torch.isfinite(o2[2, 0]).all()
        b.q = sound
        for row in ((1, 3), (2, 0)):
            o2[row], lse2[row] = o[row], lse[row]
        b.check(o2, lse2)


def test_window_slides_over_reused_pages(gpu_lib):
    """A long chat in a cache that holds no more than its window: the pages behind the
    window take the new tokens, the table says -1 for them, and every step is what
    attention over a cache of everything gives."""
    say("window reuse")
    hq, hkv, d, page, window, sinks, total = 8, 2, 64, 32, 70, 4, 400
    own = 1 + -(-window // page) + 1  # the sinks' page, and what a window can touch
    small, big = gpu_lib.Kv4Cache(own, page, hkv, d), gpu_lib.Kv4Cache(-(-total // page), page, hkv, d)
    k, v = make_kv(total, hkv, d, torch.float16, 670)
    q = randn(total, hq, d, seed=671).half().to(DEV)
    k, v = k.to(DEV), v.to(DEV)
    free, table = list(range(own)), np.full(-(-total // page), -1, np.int32)
    whole = torch.arange(-(-total // page), dtype=torch.int32, device=DEV).view(1, -1)
    for t in range(total):
        if t % page == 0:
            behind = (t - window + 1) // page  # pages before it are behind the window
            for p in range(1, max(1, behind)):
                if table[p] >= 0:
                    free.append(int(table[p]))
                    table[p] = -1
            table[t // page] = free.pop(0)
        slot = torch.tensor([int(table[t // page]) * page + t % page], device=DEV)
        gpu_lib.kv4_write(small, k[t:t + 1], v[t:t + 1], slot)
        gpu_lib.kv4_write(big, k[t:t + 1], v[t:t + 1], torch.tensor([t], device=DEV))
        lens = torch.tensor([t + 1], dtype=torch.int32, device=DEV)
        args = dict(max_kv=total, want_lse=True, window=window, sinks=sinks)
        o, lse = gpu_lib.kv4_attn(small, q[t:t + 1], torch.from_numpy(table).to(DEV)[None], lens, **args)
        o2, lse2 = gpu_lib.kv4_attn(big, q[t:t + 1], whole, lens, **args)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), t
    assert torch.isfinite(o).all()


def test_on_another_stream_and_together(gpu_lib):
    """Two streams at once, each with calls of its own inputs, outputs and workspace,
    against the same calls one after another."""
    say("two streams")
    n, hq, hkv, d = 300, 8, 2, 64
    batches = [WindowBatch(gpu_lib, [n], [900 + 100 * i], hq, hkv, d, 32, torch.float16, 680 + i, 200, 4) for i in range(2)]
    rows = [norm_inputs(64, 2048, torch.float16, torch.float32, 690 + i) for i in range(2)]
    gates = [randn(64, 4096, seed=700 + i).half().to(DEV) for i in range(2)]
    qs = [b.q.to(DEV) for b in batches]

    def calls(i):
        b = batches[i]
        res = list(gpu_lib.kv4_attn(b.cache, qs[i], b.table, b.lens, cu_q=b.cu, max_q=n, want_lse=True, window=200, sinks=4))
        res += list(gpu_lib.rms_norm_quant(rows[i][0], rows[i][2], residual=rows[i][1]))
        res += list(gpu_lib.gated_quant(gates[i][:, :2048], gates[i][:, 2048:]))
        return res
    want = [calls(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [None, None]
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = calls(i)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(want[i], got[i]))


def test_rows_past_32_bits(gpu_lib):
    """Rows whose offsets pass 2^32 bytes (a row stride, not a size), in every buffer."""
    say("row offsets")
    k, ld, m = 64, 1 << 30, 5
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of GPU memory")
    wide = torch.zeros((m - 1) * ld + k, dtype=torch.float16, device=DEV)
    qw = torch.zeros((m - 1) * ld + k, dtype=torch.int8, device=DEV)
    x, q = wide.as_strided((m, k), (ld, 1)), qw.as_strided((m, k), (ld, 1))
    x.copy_(randn(m, k, seed=720).to(DEV))
    r = torch.zeros((m - 1) * ld + k, dtype=torch.float32, device=DEV).as_strided((m, k), (ld, 1))
    r.copy_(randn(m, k, seed=721).to(DEV))
    w = torch.ones(k, device=DEV)
    _, s, _ = check_norm(gpu_lib, x, r, w, q_out=q, residual_out=r)
    check_gated(gpu_lib, x, x, "silu", q_out=q)
    torch.cuda.synchronize()
    assert not wide[k:ld].any() and not qw[k:ld].any()


@pytest.mark.parametrize("k", [64, 1001, 40000])
def test_norm_of_zeros_without_eps(gpu_lib, k):
    """A row of zeros stays zeros with eps 0, among others that do not."""
    say("zeros without eps", k)
    x = randn(3, k, seed=730).to(DEV)
    x[1] = 0
    q, s, _ = gpu_lib.rms_norm_quant(x, torch.ones(k, device=DEV), eps=0.0)
    torch.cuda.synchronize()
    assert not q[1].any() and s[1] == 1 and q[0].any() and q[2].any()


@pytest.mark.parametrize("k", [256, 2048, 8192, 1001])
def test_codes_at_ties(gpu_lib, k):
    """Quotients at and next to halves: y / s = n + 1/2 exactly, and one unit of y to
    either side (weights 1, a = 1 by choice of the row, scale 1 by its largest)."""
    say("ties", k)
    half = np.arange(-126, 126) + 0.5
    steps = np.stack([half, np.nextafter(half.astype(np.float32), np.float32(200)), np.nextafter(half.astype(np.float32), np.float32(-200))])
    vals = steps.astype(np.float32).reshape(-1)
    g = np.zeros((4, k), np.float32)
    for i in range(4):
        part = vals[i * (k - 1):(i + 1) * (k - 1)] if k < 800 else vals
        g[i, 1:1 + len(part)] = part
        g[i, 0] = 127.0
    # silu of a gate of 256 is 256 itself, and powers of two leave y = g exact
    up = torch.from_numpy(g).to(DEV)
    q, s = gpu_lib.gated_quant(torch.full((4, k), 256.0, device=DEV), up / 256)
    torch.cuda.synchronize()
    assert (s == 1).all()
    assert np.array_equal(host(q), np.clip(np.rint(g), -127, 127).astype(np.int8))
    q2, s2 = gpu_lib.act_quant(up)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("m,k", [(300, 520), (9, 2056), (40, 6152), (5, 20000)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_in_place_with_idle_threads(gpu_lib, m, k, dtype):
    """Rows shorter than their threads' runs, the residual in place, many times over."""
    say("in place, idle threads", m, k, dtype)
    x, r, w = norm_inputs(m, k, torch.float16, dtype, 740)
    want = gpu_lib.rms_norm_quant(x, w, residual=r)
    for _ in range(20):
        mine = r.clone()
        got = gpu_lib.rms_norm_quant(x, w, residual=mine, residual_out=mine)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("n,hq,d", [(2100, 33, 64), (1030, 41, 128), (5, 3, 64)])
def test_append_in_place(gpu_lib, n, hq, d):
    """q rotated where it lies, two heads a lane with one left over, many times over."""
    say("append in place", n, hq, d)
    q, k, v, cos, sin, pos, w = append_inputs(n, hq, 2, d, d, torch.float16, True, 750)
    slots = torch.arange(n, device=DEV)
    caches = [gpu_lib.Kv4Cache(n // 32 + 1, 32, 2, d) for _ in range(2)]
    want = gpu_lib.kv4_append(caches[0], q, k, v, cos, sin, pos, slots, q_weight=w[0], k_weight=w[1])
    for _ in range(20):
        mine = q.clone()
        gpu_lib.kv4_append(caches[1], mine, k, v, cos, sin, pos, slots, q_weight=w[0], k_weight=w[1], q_out=mine)
        assert torch.equal(mine, want) and torch.equal(caches[0].data, caches[1].data)


@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (128, 128, False), (64, 16, False), (128, 96, True)])
@pytest.mark.parametrize("n,hq,hkv", [(1030, 6, 3), (1400, 40, 10), (7, 3, 2), (250, 9, 1)])
def test_append_scattered(gpu_lib, d, rot, inter, n, hq, hkv):
    """Many tokens to slots in no order, of large pages, some out of range: what is
    written between them stays."""
    say("append scattered", d, rot, inter, n, hq, hkv)
    q, k, v, cos, sin, pos, w = append_inputs(n, hq, hkv, d, rot, torch.float16, True, 760 + d + n)
    cap = 256 * 8
    slots = torch.from_numpy(HOW["skips"](n, cap, np.random.default_rng(n + d)).astype(np.int64)).to(DEV)
    caches = [gpu_lib.Kv4Cache(8, 256, hkv, d) for _ in range(2)]
    for c in caches:
        c.data.fill_(0xA5)
    got = gpu_lib.kv4_append(caches[0], q, k, v, cos, sin, pos, slots, q_weight=w[0], k_weight=w[1], interleaved=inter)
    want = two_calls(gpu_lib, caches[1], q, k, v, cos, sin, pos, slots, w, inter, torch.float16)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(caches[0].data, caches[1].data)


# ------------------------------------- rows of lengths and places of any kind ---

LOOSE_SIZES = [8, 9, 12, 15, 17, 510, 513, 519, 1025, 2047, 2052, 4095, 4097, 8191, 8193, 16385, 32767]


@pytest.mark.parametrize("k", LOOSE_SIZES)
@pytest.mark.parametrize("x_dt,r_dt", [(torch.float16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                       (torch.float32, torch.float16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("first", [0, 1, 5])
def test_norm_any_place(gpu_lib, k, x_dt, r_dt, first):
    """Odd lengths from an odd place on, the residual in place, what lies around left."""
    say("norm any place", k, x_dt, r_dt, first)
    m, ld = 5, k + first + 2
    x, r, w = norm_inputs(m, k, x_dt, r_dt, 1200 + k + first)
    want = gpu_lib.rms_norm_quant(x.contiguous(), w, residual=r)
    wide = torch.full((m, ld), 55.0, device=DEV).to(r_dt)
    mine, xin = wide[:, first:first + k], torch.full((m, ld), 9.0, device=DEV).to(x_dt)[:, first:first + k]
    mine.copy_(r)
    xin.copy_(x)
    w_in = torch.ones(k + first, device=DEV)[first:]
    w_in.copy_(w)
    q_wide = torch.full((m, ld), 77, dtype=torch.int8, device=DEV)
    got = check_norm(gpu_lib, xin, mine, w_in, q_out=q_wide[:, first:first + k], residual_out=mine)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert (wide[:, :first] == 55).all() and (wide[:, first + k:] == 55).all()
    assert (q_wide[:, :first] == 77).all() and (q_wide[:, first + k:] == 77).all()


@pytest.mark.parametrize("m,k", [(2000, 513), (900, 2047), (300, 4097), (90, 16385)])
@pytest.mark.parametrize("r_dt", [torch.float16, torch.float32])
def test_norm_in_place_many_times(gpu_lib, m, k, r_dt):
    """The waves of a row, whose last runs overlap, in any order."""
    say("norm in place many times", m, k, r_dt)
    x, r, w = norm_inputs(m, k, torch.float16, r_dt, 1300 + k)
    want = gpu_lib.rms_norm_quant(x, w, residual=r)
    for _ in range(10):
        mine = r.clone()
        got = gpu_lib.rms_norm_quant(x, w, residual=mine, residual_out=mine)
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("k", LOOSE_SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("first", [0, 1, 5])
def test_gated_any_place(gpu_lib, k, dtype, first):
    say("gated any place", k, dtype, first)
    m = 5
    gu = (randn(m, 2 * k + first, seed=1400 + k) * 2).to(dtype).to(DEV)
    q_wide = torch.full((m, k + first + 2), 77, dtype=torch.int8, device=DEV)
    g, u = gu[:, first:first + k], gu[:, first + k:]
    q, s = check_gated(gpu_lib, g, u, "silu", q_out=q_wide[:, first:first + k])
    q2, s2 = gpu_lib.gated_quant(g.contiguous(), u.contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert (q_wide[:, :first] == 77).all() and (q_wide[:, first + k:] == 77).all()


@pytest.mark.parametrize("k", [1032, 1536, 2072, 3064, 4104, 6144, 6152, 12288, 12296, 24576, 24584])
@pytest.mark.parametrize("m", [1, 300])
def test_rows_aligned_shapes(gpu_lib, k, m):
    """Aligned rows on both sides of where a row gets more threads."""
    say("rows aligned shapes", k, m)
    check_norm(gpu_lib, *norm_inputs(m, k, torch.bfloat16, torch.float16, 1500 + k))
    gu = randn(m, 2 * k, seed=1600 + k).half().to(DEV)
    check_gated(gpu_lib, gu[:, :k], gu[:, k:], "gelu_tanh")


@pytest.mark.parametrize("hq,hkv,d,n,length", [(32, 8, 64, 1100, 2700), (8, 2, 64, 60, 4500), (8, 2, 128, 40, 4500),
                                               (6, 2, 128, 40, 2200)])
def test_window_many_pages(gpu_lib, hq, hkv, d, n, length):
    """Many rows over more blocks than page numbers are held at a time, in one split."""
    say("window many pages", hq, hkv, d, n, length)
    b = WindowBatch(gpu_lib, [n], [length], hq, hkv, d, 32, torch.bfloat16, 800 + d, length - n - 70, 40)
    b.check(*b.run(max_kv=100))


@pytest.mark.parametrize("hq,hkv,d,n,length", [(32, 8, 64, 1100, 1400), (8, 2, 64, 70, 200), (8, 2, 128, 70, 200)])
@pytest.mark.parametrize("power", [20, 26, 40])
def test_window_many_rows_huge_scores(gpu_lib, hq, hkv, d, n, length, power):
    """Scores that fp32 has only to units and more: every row keeps a sum and finite
    values between the least and the largest of V; rows of ordinary size among them
    stay within their bound."""
    say("window huge scores", hq, hkv, d, n, length, power)
    b = WindowBatch(gpu_lib, [n], [length], hq, hkv, d, 32, torch.bfloat16, 820 + d, 100, 4)
    o, lse = b.run()
    b.check(o, lse)
    sound = b.q.clone()
    big = torch.arange(n, device=b.q.device) % 5 == 2
    b.q[big] *= 2.0 ** power
    o2, lse2 = b.run()
    torch.cuda.synchronize()
    gpu_big = big.to(o2.device)
    assert torch.isfinite(o2).all() and torch.isfinite(lse2).all()
    vd, vround, _ = b.vd[0]
    top = float(np.abs(vd).max() + np.abs(vround).max()) * (1 + 2.0 ** -7)
    assert o2[gpu_big].abs().max().item() <= top
    b.q = sound
    o2[gpu_big], lse2[gpu_big] = o[gpu_big], lse[gpu_big]
    b.check(o2, lse2)
