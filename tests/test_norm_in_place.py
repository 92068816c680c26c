"""The residual's sum written over x: as into memory of its own, bit for bit; over x of
another type or row stride it is refused."""
import pytest
import torch

from tests.test_attn_gpu import DEV, say
from tests.test_layer_gpu import DTYPES, norm_inputs
from ultra_bit_weight_amd import sherry


def test_binding_refuses_x_of_another_shape():
    wide, w = torch.zeros(4 * 64 + 64), torch.ones(64)
    x, r = wide[:256].view(4, 64), torch.zeros(4, 64)
    with pytest.raises(ValueError, match="on the GPU"):
        sherry.rms_norm_quant(x, w, residual=r, residual_out=x)
    with pytest.raises(ValueError, match="x does, with another row stride"):
        sherry.rms_norm_quant(x, w, residual=r, residual_out=wide.view(4, 80)[:, :64])
    half = wide.view(torch.float16)
    with pytest.raises(ValueError, match="x does, with another row stride or dtype"):
        sherry.rms_norm_quant(half[:256].view(4, 64), w, residual=r, residual_out=x)
    with pytest.raises(ValueError, match="on the GPU"):  # (of one row the stride says nothing)
        sherry.rms_norm_quant(x[:1], w, residual=r[:1], residual_out=wide.view(4, 80)[:1, :64])


def test_no_rows_overlap_nothing():
    """Tensors of no rows lie nowhere, all of them: types and strides may differ."""
    w, x, r = torch.ones(64), torch.zeros(0, 64).half(), torch.zeros(0, 64)
    with pytest.raises(ValueError, match="on the GPU"):
        sherry.rms_norm_quant(x, w, residual=r, residual_out=torch.zeros(0, 64))


@pytest.mark.gpu
@pytest.mark.parametrize("m,k", [(3, 5), (300, 520), (2000, 513), (9, 2056), (90, 16385), (40, 40001)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sum_over_x(gpu_lib, m, k, dtype):
    """Short rows, aligned ones, a last run that lies over the one before, rows past the
    registers; many times over."""
    say("sum over x", m, k, dtype)
    x, r, w = norm_inputs(m, k, dtype, dtype, 750, pad=3)
    want = gpu_lib.rms_norm_quant(x, w, residual=r)
    for _ in range(10):
        mine = torch.empty(m, k + 3, dtype=dtype, device=DEV)[:, :k].copy_(x)
        got = gpu_lib.rms_norm_quant(mine, w, residual=r, residual_out=mine)
        assert got[2] is mine
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_no_rows(gpu_lib):
    say("no rows")
    x, r = torch.zeros(0, 64, device=DEV).half(), torch.zeros(0, 64, device=DEV)
    q, s, ro = gpu_lib.rms_norm_quant(x, torch.ones(64, device=DEV), residual=r)
    assert q.shape == (0, 64) and s.shape == (0,) and ro.shape == (0, 64) and ro.dtype == torch.float32
