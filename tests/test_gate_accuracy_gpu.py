"""What include/sherry.h says of the gated activation's accuracy, value by value, and
codes that reach 127 in every row."""
import numpy as np
import pytest
import torch

from oracle import layer_ref
from tests.test_attn_gpu import DEV, host, randn, say

pytestmark = pytest.mark.gpu


def z_of(g, act):
    return g if act == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)


def stated_bound(g, u, act):
    """include/sherry.h: (10 + c max(0, -z)) 2^-24 of the value, c 2 or 7, and 2^-119 |up|.
    Half steps of fp32: the exponential's own step 2, its sum with 1 1, the reciprocal 2,
    two products 2; of its argument |z| times the rounding of z log2 e and of the
    constant, 1.3; of GELU's z besides two products (3 + 0.6) for the cube's share of it
    (0.82 where exp passes fp32), the sum, the product and its constant 2.5, 6.7 in all.  For z > 0
    the exponential's error counts by its share z exp(-z) / (1 + exp(-z)) < 0.28: 2 more
    at most.  Beyond exp(-z) = 2^126 the reciprocal is below the normal numbers: nothing,
    of a value below 89 * 2^-126."""
    y = np.abs(layer_ref.gated(g, u, act))
    return y * (10 + (2 if act == "silu" else 7) * np.maximum(0, -z_of(g, act))) * 2.0 ** -24 + 2.0 ** -119 * np.abs(u) + 2.0 ** -149


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("k", [3, 16, 1001])
@pytest.mark.parametrize("up", [1.0, -3.7e-5, 2.0 ** 60])
def test_gate_accuracy(gpu_lib, act, k, up):
    """One gate a row, so that the row's scale is its value over 127."""
    say("gate accuracy", act, k, up)
    rng = np.random.default_rng(5)
    far = 95.0 if act == "silu" else 11.0
    g = np.concatenate([rng.uniform(-far, far, 6000), rng.uniform(-3, 3, 1000), 10.0 ** rng.uniform(-38, 12, 500),
                        -(10.0 ** rng.uniform(-38, 12, 500)), [0.0, -0.0]]).astype(np.float32)
    u = np.full(g.shape, up, np.float32)
    wide = torch.from_numpy(np.repeat(g[:, None], k, 1)).to(DEV)
    q, s = gpu_lib.gated_quant(wide, torch.full_like(wide, float(u[0])), activation=act)
    torch.cuda.synchronize()
    g, u = g.astype(np.float64), u.astype(np.float64)
    y = np.abs(layer_ref.gated(g, u, act))
    got = host(s).astype(np.float64) * 127
    none = got == 127  # (a scale of 1: a row of zeros)
    got = np.where(none & (y < 100), 0, got)
    off = np.abs(got - y)
    bound = stated_bound(g, u, act)
    units = off / np.maximum(y, 2.0 ** -126) * 2.0 ** 23
    for lo, hi in ((-95, -40), (-40, -20), (-20, -10), (-10, -5), (-5, -1), (-1, 1), (1, 100)):
        at = (g >= lo) & (g < hi) & (y > 2.0 ** -110 * np.abs(u))
        if at.any():
            say(f"   g in [{lo}, {hi}): off by up to {units[at].max():.1f} units, {(off / bound)[at].max():.3f} of the bound")
    assert (off <= bound * (1 + 2.0 ** -20) + (y + bound) * 2.0 ** -24 + 127 * 2.0 ** -150).all(), np.flatnonzero(off > bound)[:5]
    q, s = host(q).astype(np.int64), host(s)
    assert not q[none].any() and (np.abs(q[~none & (s >= 2.0 ** -126)]) == 127).all()


@pytest.mark.parametrize("k", [7, 512, 1001, 40000])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_every_gated_row_reaches_127(gpu_lib, k, act):
    """Large, tiny and ordinary rows beside rows of zeros: the largest value of each has
    the code 127, zeros have 0 and the scale 1."""
    say("gated rows reach 127", k, act)
    g, u = randn(9, k, seed=1), randn(9, k, seed=2)
    g[1] = 0
    u[2] = 0
    u[3] *= 1e30
    u[4] *= 1e-30
    g[5] *= 1e-20
    g[6] = g[6] * 10 + 40
    u[7, 1:] = 0
    q, s = gpu_lib.gated_quant(g.to(DEV), u.to(DEV), activation=act)
    torch.cuda.synchronize()
    q, s = host(q).astype(np.int64), host(s)
    zero = np.isin(np.arange(9), [1, 2])
    assert (np.abs(q).max(-1)[~zero] == 127).all() and np.isfinite(s).all() and (s[~zero] != 1).all()
    assert not q[zero].any() and (s[zero] == 1).all()
