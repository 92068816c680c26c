"""CPU reference of the attention operators (numpy, fp64): the 4-bit key/value
cache's quantiser and byte layout, norms with rotation, causal attention over a
cache.  Written from the definitions in include/sherry.h; shares no code with
the library.

Readings: A1 the quantiser's steps are IEEE fp32 (difference, one division,
round half to even), its scale and zero point fp16; A2 a cached value stands
for z + s c; A3 token i of n new ones sees cached tokens 0 .. L - n + i; A4 a
row that sees nothing is zeros, its log-sum -inf.
"""
import numpy as np

GROUP, BLOCK = 64, 32
F16_MAX = 65504.0


def quantise(x):
    """x [..., D] of fp32-exact values -> codes uint8 [..., D], s, z fp16 [..., D/64]"""
    x = np.asarray(x, np.float32)
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    lo, hi = y.min(-1), y.max(-1)
    z = np.clip(lo, -F16_MAX, F16_MAX).astype(np.float16)
    with np.errstate(over="ignore"):
        s = np.minimum(((hi - lo) / np.float32(15)).astype(np.float32), np.float32(F16_MAX)).astype(np.float16)
        s32 = s.astype(np.float32)[..., None]
        t = (y - z.astype(np.float32)[..., None]).astype(np.float32)
        r = np.rint((t / np.where(s32 > 0, s32, np.float32(1))).astype(np.float32))
    c = np.where(s32 > 0, np.clip(r, 0, 15), 0).astype(np.uint8)
    return c.reshape(x.shape), s, z


def dequantise(c, s, z):
    """fp64 values z + s c (exact)."""
    y = c.reshape(c.shape[:-1] + (c.shape[-1] // GROUP, GROUP)).astype(np.float64)
    return (z.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * y).reshape(c.shape)


def block_bytes(d):
    return 32 * d + 256 * (d // GROUP)


B = (0, 2, 1, 3)


def k_byte(d, t, i):
    """(byte of the block, shift) of K value i of token t"""
    r, h, j = i // 64, i % 64 // 8, i % 8
    tile = t // 16
    if d == 64:
        at = ((h % 4 * 16 + t % 16) * 2 + tile) * 8
    else:
        at = ((tile * 4 + h % 4) * 16 + t % 16) * 16 + 8 * r
    return at + j // 4 * 4 + B[j % 4], 0 if h < 4 else 4


def v_byte(d, t, i):
    p, e = i // 32, i % 16
    g, tile = t % 16 // 4, t // 16
    return 16 * d + p // 2 * 1024 + (g * 16 + e) * 16 + p % 2 * 8 + tile * 4 + B[t % 4], 4 if i % 32 >= 16 else 0


def scale_byte(d, t, r, w):
    return 32 * d + 256 * r + 64 * w + 16 * (t % 16 // 4) + 8 * (t // 16) + 2 * (t % 4)


def store(data, page_size, n_heads, slot, head, kc, ks, kz, vc, vs, vz):
    """One token's codes and scales into the cache's bytes (uint8 [bytes])."""
    d = kc.size
    page, place = divmod(slot, page_size)
    blk = ((page * n_heads + head) * (page_size // BLOCK) + place // BLOCK) * block_bytes(d)
    t = place % BLOCK
    for c, where in ((kc, k_byte), (vc, v_byte)):
        for i in range(d):
            at, sh = where(d, t, i)
            data[blk + at] = (int(data[blk + at]) & (0xF0 if sh == 0 else 0x0F)) | (int(c[i]) << sh)
    for r in range(d // GROUP):
        for w, a in enumerate((ks, kz, vs, vz)):
            at = blk + scale_byte(d, t, r, w)
            data[at:at + 2] = np.frombuffer(np.float16(a[r]).tobytes(), np.uint8)


def norm_rope(x, w, cos, sin, eps, rot, interleaved):
    """x [n, heads, d], cos / sin [n, rot/2] of each token's position -> fp64"""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y = x.copy()
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    c, s = (np.asarray(t, np.float64)[:, None, :] for t in (cos, sin))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def attention(q, k, v, scale, vmag=None):
    """One sequence: q [n, hq, d], k and v [L, hkv, d] -> out fp64 [n, hq, d],
    lse [n, hq], and sum_j w_j vmag_j [n, hq, d] (vmag: |v| unless given; what
    errors of the terms scale with)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    vmag = np.abs(v) if vmag is None else vmag
    n, hq, d = q.shape
    length, hkv = k.shape[:2]
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    for h in range(hq):
        kh = h // (hq // hkv)
        for i in range(n):
            seen = max(0, min(length, length - n + i + 1))
            if seen == 0:
                continue
            s = scale * (k[:seen, kh] @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            lse[i, h] = m + np.log(e.sum())
            out[i, h] = e @ v[:seen, kh] / e.sum()
            mag[i, h] = e @ vmag[:seen, kh] / e.sum()
    return out, lse, mag
