"""Planted mistakes in a private copy of the attention reference must trip at
least one of its pins (tests/test_attn_oracle.py)."""
import os
import types

import pytest

from tests import test_attn_oracle as pins

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "oracle", "attn_ref.py")
PINS = [pins.test_quantiser_by_hand, pins.test_quantiser_error_bound, pins.test_quantiser_steps_by_fractions,
        pins.test_quantiser_extremes, lambda: pins.test_layout_is_a_bijection(64),
        lambda: pins.test_layout_is_a_bijection(128), pins.test_layout_by_hand, pins.test_store_keeps_neighbours,
        pins.test_rotation_closed_forms, pins.test_attention_closed_forms]
MUTANTS = {
    "sixteen_steps": ("/ np.float32(15)", "/ np.float32(16)"),
    "zero_at_the_top": ("z = np.clip(lo,", "z = np.clip(hi,"),
    "codes_truncated": ("r = np.rint(", "r = np.trunc("),
    "half_away_from_zero": ("r = np.rint((t / np.where(s32 > 0, s32, np.float32(1))).astype(np.float32))",
                            "r = np.floor((t / np.where(s32 > 0, s32, np.float32(1))).astype(np.float32) + np.float32(0.5))"),
    "scale_not_clamped": ("s = np.minimum(((hi - lo) / np.float32(15)).astype(np.float32), np.float32(F16_MAX))",
                          "s = ((hi - lo) / np.float32(15)).astype(np.float32)"),
    "zero_point_dropped": ("z.astype(np.float64)[..., None] + s", "0 * z.astype(np.float64)[..., None] + s"),
    "bytes_in_order": ("B = (0, 2, 1, 3)", "B = (0, 1, 2, 3)"),
    "k_nibbles_swapped": ("B[j % 4], 0 if h < 4 else 4", "B[j % 4], 4 if h < 4 else 0"),
    "v_halves_swapped": ("B[t % 4], 4 if i % 32 >= 16 else 0", "B[t % 4], 0 if i % 32 >= 16 else 4"),
    "v_tiles_overlap": ("p % 2 * 8 + tile * 4", "p % 2 * 8"),
    "rotation_backwards": ("y[..., a] = x[..., a] * c - x[..., b] * s", "y[..., a] = x[..., a] * c + x[..., b] * s"),
    "mean_not_square": ("np.sqrt((x * x).mean(-1, keepdims=True) + eps)", "np.sqrt(np.abs(x).mean(-1, keepdims=True) + eps)"),
    "one_token_early": ("min(length, length - n + i + 1)", "min(length, length - n + i)"),
    "one_token_late": ("min(length, length - n + i + 1)", "min(length, length - n + i + 2)"),
    "heads_interleaved": ("kh = h // (hq // hkv)", "kh = h % hkv"),
    "scale_after_softmax": ("s = scale * (k[:seen, kh] @ q[i, h])", "s = k[:seen, kh] @ q[i, h]"),
    "lse_without_maximum": ("lse[i, h] = m + np.log(e.sum())", "lse[i, h] = np.log(e.sum())"),
}


def fresh(patch=None):
    src = open(PATH).read()
    if patch:
        assert patch[0] in src, patch[0]
        src = src.replace(patch[0], patch[1])
    mod = types.ModuleType("attn_ref_planted")
    exec(compile(src, PATH, "exec"), mod.__dict__)
    return mod


def caught_by(mod, monkeypatch):
    monkeypatch.setattr(pins, "attn_ref", mod)
    n = 0
    for pin in PINS:
        try:
            pin()
        except (AssertionError, ValueError, OverflowError, FloatingPointError, IndexError):
            n += 1
    return n


def test_copy_passes_every_pin(monkeypatch):
    assert caught_by(fresh(), monkeypatch) == 0


@pytest.mark.parametrize("name", sorted(MUTANTS))
def test_planted_mistake_is_caught(name, monkeypatch):
    assert caught_by(fresh(MUTANTS[name]), monkeypatch), f"{name} passed every pin"
