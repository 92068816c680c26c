"""Pins of the attention reference (oracle/attn_ref.py) against facts from
outside it: hand-worked codes, hand-placed bytes, closed forms."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import attn_ref


def test_quantiser_by_hand():
    """0..15 in steps of a power of two: scale 1/4, zero -1, codes 0..15; a
    constant group has scale 0 and codes 0; ties go to even."""
    x = np.zeros((3, 64), np.float32)
    x[0] = -1 + 0.25 * (np.arange(64) % 16)
    x[1] = 3.5
    x[2, 0], x[2, 1], x[2, 2], x[2, 3], x[2, 4] = 0, 15, 0.5, 1.5, 2.5
    c, s, z = attn_ref.quantise(x)
    assert s[0, 0] == 0.25 and z[0, 0] == -1 and np.array_equal(c[0], np.arange(64) % 16)
    assert s[1, 0] == 0 and z[1, 0] == 3.5 and not c[1].any()
    assert s[2, 0] == 1 and list(c[2, :5]) == [0, 15, 0, 2, 2]
    assert np.array_equal(attn_ref.dequantise(c, s, z)[:2], x[:2])


def test_quantiser_error_bound():
    """Every value within half a step, plus what the rounded zero point and
    scale add (fp16: 2^-11 of each)."""
    x = (np.random.default_rng(1).standard_normal((50, 128)) * 3).astype(np.float32)
    c, s, z = attn_ref.quantise(x)
    assert c.min() == 0 and c.max() == 15
    err = np.abs(attn_ref.dequantise(c, s, z) - x).reshape(50, 2, 64)
    bound = s.astype(np.float64) * (0.5 + 15 * 2.0 ** -11) + np.abs(z.astype(np.float64)) * 2.0 ** -11
    assert (err <= bound[..., None] * (1 + 1e-6)).all()


def test_quantiser_steps_by_fractions():
    """Codes against exact rationals rounded as the definition says (to fp32
    after the difference and after the quotient)."""
    def f32(v):
        return Fraction(float(np.float32(float(v)))) if v else Fraction(0)
    x = (np.random.default_rng(2).standard_normal((4, 64)) * 10).astype(np.float16).astype(np.float32)
    c, s, z = attn_ref.quantise(x)
    for r in range(4):
        fs, fz = Fraction(float(s[r, 0])), Fraction(float(z[r, 0]))
        for i in range(64):
            t = f32(Fraction(float(x[r, i])) - fz)
            quo = f32(t / fs)
            assert min(max(round(quo), 0), 15) == c[r, i]  # round(): half to even


def test_quantiser_extremes():
    """Beyond fp16: scale and zero point stay finite; infinitely wide ranges too."""
    x = np.zeros((2, 64), np.float32)
    x[0, 0], x[0, 1] = -3e38, 3e38
    x[1, 0], x[1, 1] = -1e5, 1e-8
    c, s, z = attn_ref.quantise(x)
    assert np.isfinite(s.astype(np.float64)).all() and np.isfinite(z.astype(np.float64)).all()
    assert s[0, 0] == 65504 and z[0, 0] == -65504 and c[0, 0] == 0 and c[0, 1] == 15


@pytest.mark.parametrize("d", [64, 128])
def test_layout_is_a_bijection(d):
    """Every nibble of a block's code bytes belongs to one value of K or V, and
    every scale byte to one parameter."""
    seen = set()
    for t in range(32):
        for i in range(d):
            for where in (attn_ref.k_byte, attn_ref.v_byte):
                at = where(d, t, i)
                assert at not in seen and 0 <= at[0] < 32 * d
                seen.add(at)
    assert len(seen) == 2 * 32 * d
    scales = {attn_ref.scale_byte(d, t, r, w) for t in range(32) for r in range(d // 64) for w in range(4)}
    assert len(scales) == 32 * d // 64 * 4 and min(scales) == 32 * d
    assert max(scales) + 2 == attn_ref.block_bytes(d)


def test_layout_by_hand():
    """Places worked out by hand from the description in the header."""
    assert attn_ref.k_byte(64, 0, 0) == (0, 0)
    assert attn_ref.k_byte(64, 0, 1) == (2, 0)       # B(1) = 2
    assert attn_ref.k_byte(64, 0, 32) == (0, 4)      # h = 4: high nibble
    assert attn_ref.k_byte(64, 17, 8) == (((16 + 1) * 2 + 1) * 8, 0)
    assert attn_ref.k_byte(128, 17, 64 + 13) == (((4 + 1) * 16 + 1) * 16 + 8 + 4 + 2, 0)
    assert attn_ref.v_byte(64, 0, 0) == (1024, 0) and attn_ref.v_byte(64, 0, 16) == (1024, 4)
    assert attn_ref.v_byte(64, 22, 37) == (1024 + (16 + 5) * 16 + 8 + 4 + 1, 0)
    assert attn_ref.v_byte(128, 0, 64) == (2048 + 1024, 0)
    assert attn_ref.scale_byte(128, 22, 1, 3) == 4096 + 256 + 192 + 16 + 8 + 4


def test_store_keeps_neighbours():
    d = 64
    data = np.full(attn_ref.block_bytes(d) * 2, 0xA5, np.uint8)
    c = np.arange(64, dtype=np.uint8) % 16
    one = np.array([1.0], np.float16)
    attn_ref.store(data, 32, 1, 33, 0, c, one, one, c, one, one)
    assert (data[:attn_ref.block_bytes(d)] == 0xA5).all()
    touched = {attn_ref.k_byte(d, 1, i)[0] for i in range(d)} | {attn_ref.v_byte(d, 1, i)[0] for i in range(d)}
    touched |= {attn_ref.scale_byte(d, 1, 0, w) + b for w in range(4) for b in (0, 1)}
    base = attn_ref.block_bytes(d)
    assert all(data[base + i] == 0xA5 for i in range(base) if i not in touched)
    assert len(touched) == 32 + 32 + 8


def test_rotation_closed_forms():
    """A quarter turn swaps the pair's values; any turn keeps their norm; unit
    weights make the mean square 1; partial rotation leaves the rest."""
    x = np.random.default_rng(3).standard_normal((2, 3, 32))
    one, zero = np.ones((2, 8)), np.zeros((2, 8))
    for inter, (a, b) in ((False, (0, 8)), (True, (0, 1))):
        y = attn_ref.norm_rope(x, None, zero, one, 0.0, 16, inter)
        assert np.array_equal(y[..., a], -x[..., b]) and np.array_equal(y[..., b], x[..., a])
        assert np.array_equal(y[..., 16:], x[..., 16:])
    th = np.random.default_rng(4).uniform(0, 6, (2, 8))
    y = attn_ref.norm_rope(x, None, np.cos(th), np.sin(th), 0.0, 16, True)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-13)
    y = attn_ref.norm_rope(x, np.ones(32), one, zero, 0.0, 16, False)
    assert np.allclose((y ** 2).mean(-1), 1, rtol=1e-13)


def test_attention_closed_forms():
    """Equal keys average the visible values; one visible token is returned; a
    row that sees nothing is zeros; a group of query heads shares a key head."""
    r = np.random.default_rng(5)
    v = r.standard_normal((6, 2, 64))
    q = r.standard_normal((3, 4, 64))
    out, lse, _ = attn_ref.attention(q, np.ones((6, 2, 64)), v, 0.5)
    for i in range(3):
        for h in range(4):
            assert np.allclose(out[i, h], v[:4 + i, h // 2].mean(0), atol=1e-14)
            assert np.isclose(lse[i, h], 0.5 * q[i, h].sum() + np.log(4 + i))
    out, lse, _ = attn_ref.attention(q, v[:2], v[:2], 1.0)
    assert not out[0].any() and np.isneginf(lse[0]).all()
    assert np.allclose(out[1, 3], v[0, 1])
