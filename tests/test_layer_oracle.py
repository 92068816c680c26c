"""Pins of the reference of the operators around a layer's products
(oracle/layer_ref.py): values by hand, by fractions, closed forms, and each
planted mistake caught."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import attn_ref, layer_ref


def test_norm_by_hand():
    """h = (3, 4): mean of squares 12.5; with weights that undo the root the codes
    are 95 (127 * 3 / 4 = 95.25) and 127."""
    q, s, h = layer_ref.rms_norm_quant([[1.0, 6.0]], [[2.0, -2.0]], [1.0, 1.0], 0.0)
    a = np.float32(1 / math.sqrt(12.5))
    assert h.tolist() == [[3.0, 4.0]] and q.tolist() == [[95, 127]]
    assert s[0] == np.float32(np.float32(np.float32(4) * a) / np.float32(127))


def test_norm_eps_zero_rows_and_signs():
    q, s, _ = layer_ref.rms_norm_quant(np.zeros((1, 8)), None, np.ones(8), 1e-6)
    assert not q.any() and s[0] == 1.0
    y, _ = layer_ref.rms_norm([[1e-3] * 4], None, np.ones(4), 1e-6)  # mean of squares = eps: 1 / sqrt(2)
    assert np.allclose(y, math.sqrt(0.5), rtol=1e-6)
    x = np.random.default_rng(0).standard_normal((3, 40)).astype(np.float32)
    q1, s1, _ = layer_ref.rms_norm_quant(x, None, np.ones(40), 1e-6)
    q2, s2, _ = layer_ref.rms_norm_quant(-x, None, np.ones(40), 1e-6)
    assert np.array_equal(q1, -q2) and np.array_equal(s1, s2)
    q3, s3, _ = layer_ref.rms_norm_quant(4 * x, None, np.ones(40), 0.0)  # a power of two cancels
    q4, s4, _ = layer_ref.rms_norm_quant(x, None, np.ones(40), 0.0)
    assert np.array_equal(q3, q4) and np.array_equal(s3, s4)


def test_norm_is_of_the_unrounded_sum():
    """1 + 2^-12 is not a bf16 or fp16 value: the norm sees it (L1)."""
    x, r = np.array([[1.0, -1.0]]), np.array([[2.0 ** -12, 0.0]])
    y, h = layer_ref.rms_norm(x, r, [1.0, 1.0], 0.0)
    assert h[0, 0] == 1 + 2.0 ** -12 and y[0, 0] / -y[0, 1] == pytest.approx(1 + 2.0 ** -12, rel=1e-7)


def test_norm_factor_by_fractions():
    """a is the fp32 number nearest the exact 1 / sqrt: its neighbours bracket it."""
    rng = np.random.default_rng(1)
    h = (rng.standard_normal(50) * 2.0 ** rng.integers(-30, 30, 50)).astype(np.float32)
    y, _ = layer_ref.rms_norm([h], None, np.ones(50), 0.0)
    a = np.float32(y[0][np.argmax(np.abs(h))] / h[np.argmax(np.abs(h))])
    mean = sum(Fraction(float(v)) ** 2 for v in h) / 50
    lo, hi = (Fraction(float(np.nextafter(a, np.float32(d)))) for d in (0, np.inf))
    assert lo * lo * mean < 1 < hi * hi * mean


def test_sum_of_squares_cancels_nothing():
    row = np.array([1e18, 1.0, 1e-18], np.float32)
    assert layer_ref.sum_of_squares(row) == float(sum(Fraction(float(v)) ** 2 for v in row))


def test_gates_closed_forms():
    g = np.linspace(-30, 30, 121)
    assert np.allclose(layer_ref.gate(g, "silu"), g * (0.5 + 0.5 * np.tanh(g / 2)), rtol=1e-9, atol=1e-12)
    gelu = 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    assert np.allclose(layer_ref.gate(g, "gelu_tanh"), gelu, rtol=1e-9, atol=1e-12)
    # silu(g) - silu(-g) = g; gelu likewise
    for act in ("silu", "gelu_tanh"):
        assert np.allclose(layer_ref.gate(g, act) - layer_ref.gate(-g, act), g, rtol=1e-12)
    assert layer_ref.gate(1.0, "silu") == pytest.approx(math.e / (1 + math.e))
    assert layer_ref.gated(2.0, -3.0, "silu") == -3 * layer_ref.gate(2.0, "silu")
    with pytest.raises(ValueError):
        layer_ref.gate(g, "relu")


def test_visible_by_hand():
    see = layer_ref.visible(3, 6, 2, 1)  # tokens at positions 3, 4, 5
    assert see.astype(int).tolist() == [[1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    assert layer_ref.visible(2, 1, 1, 0).astype(int).tolist() == [[0], [1]]
    assert layer_ref.visible(1, 4, 4, 0).all() and not layer_ref.visible(1, 4, 3, 0)[0, 0]


def test_window_of_everything_is_attention():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    for window, sinks in ((9, 0), (1, 9), (100, 100)):
        for x, y in zip(layer_ref.window_attention(q, k, v, 0.3, window, sinks), attn_ref.attention(q, k, v, 0.3)):
            assert np.allclose(x, y, rtol=1e-12, atol=0)


def test_window_is_attention_over_what_is_left():
    """The last token with a window and sinks: attention over those tokens alone."""
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((1, 2, 8)), rng.standard_normal((20, 1, 8)), rng.standard_normal((20, 1, 8))
    at = [0, 1, 2, 15, 16, 17, 18, 19]
    for x, y in zip(layer_ref.window_attention(q, k, v, 0.3, 5, 3), attn_ref.attention(q, k[at], v[at], 0.3)):
        assert np.allclose(x, y, rtol=1e-12, atol=0)
    out, lse, _ = layer_ref.window_attention(q, k, v, 0.3, 1, 0)  # itself alone
    assert np.allclose(out[0], v[19]) and np.allclose(lse[0], 0.3 * (q[0] @ k[19, 0]))


MISTAKES = {
    "window one too wide": (layer_ref, "visible", lambda f: lambda n, length, w, s: f(n, length, w + 1, s)),
    "window one too narrow": (layer_ref, "visible", lambda f: lambda n, length, w, s: f(n, length, max(1, w - 1), s)),
    "one sink more": (layer_ref, "visible", lambda f: lambda n, length, w, s: f(n, length, w, s + 1)),
    "sinks ignored": (layer_ref, "visible", lambda f: lambda n, length, w, s: f(n, length, w, 0)),
    "rows in the opposite order": (layer_ref, "visible", lambda f: lambda n, length, w, s: f(n, length, w, s)[::-1]),
    "gate on the wrong side": (layer_ref, "gated", lambda f: lambda g, u, act: f(u, g, act)),
    "gelu as silu": (layer_ref, "gate", lambda f: lambda g, act: f(g, "silu")),
    "squares in fp32": (layer_ref, "sum_of_squares", lambda f: lambda row: float((row * row).sum(dtype=np.float32))),
    "mean left out": (layer_ref, "sum_of_squares", lambda f: lambda row: f(row) * len(row)),
}
PINS = [test_norm_by_hand, test_norm_eps_zero_rows_and_signs, test_norm_is_of_the_unrounded_sum,
        test_norm_factor_by_fractions, test_sum_of_squares_cancels_nothing, test_gates_closed_forms, test_visible_by_hand,
        test_window_of_everything_is_attention, test_window_is_attention_over_what_is_left]


@pytest.mark.parametrize("name", list(MISTAKES))
def test_planted_mistakes_are_caught(name, monkeypatch):
    where, attr, wrong = MISTAKES[name]
    monkeypatch.setattr(where, attr, wrong(getattr(where, attr)))
    caught = 0
    for pin in PINS:
        try:
            pin()
        except Exception:  # noqa: BLE001  (a pin that fails in any way has caught it)
            caught += 1
    assert caught, name
