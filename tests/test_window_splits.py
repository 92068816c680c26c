"""How a windowed call of few rows splits its sequences: by the rule that the launch
uses (kv4_attn_window_splits, no GPU needed), and its results where it splits calls that
fill the chip."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_abi_host import lib  # noqa: F401
from tests.test_attn_gpu import say
from tests.test_layer_gpu import WindowBatch


def rules(lib):  # noqa: F811
    """splits with a window and without one, of tile_rows, workgroups, tokens seen (and head_dim)"""
    window, plain = lib["_ZN6sherry22kv4_attn_window_splitsEilli"], lib["_ZN6sherry15kv4_attn_splitsEill"]
    window.restype = plain.restype = ctypes.c_int32
    plain.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int64]
    window.argtypes = [*plain.argtypes, ctypes.c_int]
    return window, plain


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tile", [8, 16])
def test_long_windows_split_as_none_does(lib, tile, d):  # noqa: F811
    """A window of nearly all that a table holds is split as the call without one, from
    one workgroup a CU on too (31 sequences of 8 heads: 7 splits, and 32: 1, it was)."""
    window, plain = rules(lib)
    for groups in [1, 3, 17, 100, 248, *range(256, 1700, 8), 4000]:
        for seen in (8192, 11000, 20000, 32764, 131072, 1 << 30):
            assert window(tile, groups, seen, d) == plain(tile, groups, seen), (groups, seen)
    assert window(tile, 320, 4096, d) == plain(tile, 320, 4096) > 1


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tile", [8, 16])
def test_short_windows_of_many_sequences_stay_whole(lib, tile, d):  # noqa: F811
    window, _ = rules(lib)
    for groups in (256, 384, 447, 448, 512, 1024, 5000):
        assert all(window(tile, groups, seen, d) == 1 for seen in (1, 100, 2052, 4000))
    assert window(tile, 480, 8000, d) == window(tile, 1024, 8000, d) == 1


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tile", [8, 16])
def test_splits_grow_with_the_tokens_seen(lib, tile, d):  # noqa: F811
    """(So that the workspace of a max_kv serves every smaller one.)"""
    window, _ = rules(lib)
    for groups in (1, 8, 100, 255, 256, 300, 447, 448, 511, 512, 800, 1535, 1536, 3000):
        n = [window(tile, groups, seen, d) for seen in [*range(1, 9000, 7), *range(9000, 200000, 999), 1 << 30]]
        assert all(a <= b for a, b in zip(n, n[1:])), groups
        assert n[-1] * groups * tile * (d + 2) * 4 <= 66 << 20 or n[-1] == 1


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d,seqs,q", [(16, 8, 64, 33, 1), (16, 16, 128, 17, 9), (24, 8, 64, 40, 4)])
def test_window_of_many_sequences_split(gpu_lib, hq, hkv, d, seqs, q):
    """Ragged sequences, some shorter than a split, at least 256 workgroups: with two
    splits and more, and by a smaller max_kv whole."""
    say("window many sequences", hq, hkv, d, seqs, q)
    rng = np.random.default_rng(5)
    ls = [int(x) for x in np.exp(rng.uniform(np.log(q + 1), np.log(3000), seqs))]
    ls[3], ls[5] = 5200, 0
    b = WindowBatch(gpu_lib, [q] * seqs, ls, hq, hkv, d, 64, torch.bfloat16, 3300 + d, 4300, 4)
    for max_kv in (max(ls), 1000, 1 << 30):
        o, lse = b.run(max_kv=max_kv)
        b.check(o, lse)
