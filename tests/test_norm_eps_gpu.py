"""Norms to int8 without eps: rows of zeros, rows that the residual cancels, and rows so
small that the factor 1 / sqrt(mean square) passes fp32, on the GPU against the CPU
reference, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import layer_ref
from tests.test_attn_gpu import DEV, host, randn, say


def test_reference_of_tiny_rows():
    """h a w with a the largest fp32: by hand, of powers of two (and zeros beside them)."""
    x = np.array([[2.0 ** -149, 0, -(2.0 ** -148), 0]], np.float32)
    w = np.array([1, 2, 4, 1], np.float32)
    q, s, h = layer_ref.rms_norm_quant(x, None, w, 0.0)
    top = np.float32(2.0 ** -18 * (1 - 2.0 ** -24))  # 2^-148 (2^128 - 2^104) 4
    assert np.array_equal(h, x) and s[0] == np.float32(top / np.float32(127))
    assert q.tolist() == [[16, 0, -127, 0]]  # an eighth of 127: 15.875


@pytest.mark.gpu
@pytest.mark.parametrize("k", [5, 64, 512, 1001, 8200, 40000])
@pytest.mark.parametrize("r_dt", [None, torch.float32, torch.bfloat16])
def test_norm_without_eps(gpu_lib, k, r_dt):
    """Rows of zeros, rows that the residual cancels, and rows so small that 1 / sqrt of
    their mean square passes fp32 (a is its largest number there), between others."""
    say("norm without eps", k, r_dt)
    x = randn(10, k, seed=8).bfloat16().float()
    x[0] = 0
    x[1] = 1e-42
    x[2] *= 2.0 ** -133
    x[3] = 0
    x[3, k // 2] = -(2.0 ** -149)
    x[4] *= 2.0 ** -126
    x[5] *= 2.0 ** -128
    r = torch.zeros(10, k)
    r[6] = -x[6]
    x[7] = 2.0 ** -149
    x, r = x.to(DEV), None if r_dt is None else r.to(r_dt).to(DEV)
    w = (1 + 0.3 * randn(k, seed=9)).to(DEV)
    q, s, ro = gpu_lib.rms_norm_quant(x, w, residual=r, eps=0.0)
    torch.cuda.synchronize()
    with np.errstate(divide="ignore", invalid="ignore"):
        rq, rs, h = layer_ref.rms_norm_quant(host(x), None if r is None else host(r.float()), host(w), 0.0)
    zeros = ~h.any(-1)
    assert zeros.sum() == (1 if r is None else 2)
    q, s = host(q), host(s)
    assert not q[zeros].any() and (s[zeros] == 1).all()
    assert np.isfinite(s).all() and np.array_equal(s[~zeros], rs[~zeros]) and np.array_equal(q[~zeros], rq[~zeros])
    assert (np.abs(q.astype(np.int64)).max(-1)[~zeros] == 127).all()
    if r is not None:
        assert np.array_equal(host(ro.float()), host(torch.from_numpy(h).to(r_dt).float()))
