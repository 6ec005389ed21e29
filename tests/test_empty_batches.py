"""Batches of no rows, as the quantizers hand them over: int8_quantize_rows returns a scale tensor
of one element for them, which the products take."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from test_operator_overlaps import F32, I8, NOT_CUDA, built, z

assert built                           # the fixture that builds the extension module


def test_scales_of_no_rows():
    one, eight = z(1, dtype=F32), z(8, dtype=F32)
    with pytest.raises(TypeError, match=NOT_CUDA):
        nv.int8_gemm_act(z(0, 64, dtype=I8), one, z(8, 64, dtype=I8), eight)
    with pytest.raises(TypeError, match=NOT_CUDA):
        nv.int8_gemm_act(z(8, 64, dtype=I8), eight, z(0, 64, dtype=I8), one)
    with pytest.raises(TypeError, match=NOT_CUDA):
        nv.int8_linear_act(z(8, 64), z(0, 64, dtype=I8), one, workspace=z(8192, dtype=torch.uint8))
    with pytest.raises(ValueError, match="sa must be"):
        nv.int8_gemm_act(z(0, 64, dtype=I8), z(2, dtype=F32), z(8, 64, dtype=I8), eight)
    with pytest.raises(ValueError, match="sa must be"):
        nv.int8_gemm_act(z(2, 64, dtype=I8), one, z(8, 64, dtype=I8), eight)
    with pytest.raises(ValueError, match="sb must be"):
        nv.int8_gemm_act(z(2, 64, dtype=I8), z(2, dtype=F32), z(8, 64, dtype=I8), one)


@pytest.mark.gpu
def test_a_block_on_no_rows():
    x = torch.zeros(0, 128, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(64, 128, device="cuda").to(torch.bfloat16)
    wq = nv.int8_quantize_rows(w)
    assert nv.int8_gemm_act(*nv.int8_quantize_rows(x), *wq, activation="gelu").shape == (0, 64)
    q, s, h = nv.int8_rmsnorm_quantize(x, None, 1e-6, residual=x)
    assert h.shape == x.shape and nv.int8_gemm_act(q, s, *wq, gated=True).shape == (0, 32)
    assert nv.int8_linear_act(x, *wq, activation="silu").shape == (0, 64)
    wp, wsf, gw = nv.pack_weight(w)
    assert nv.nvfp4_linear_act(x, wp, wsf, gw, 64, activation="silu").shape == (0, 64)
    p, sf, g = nv.nvfp4_quantize(x)
    assert nv.nvfp4_gemm_act(p, sf, wp, wsf, torch.ones(1, device="cuda"), None, 0, 64, 128).shape == (0, 64)
    none = nv.int8_quantize_rows(w[:0])
    assert nv.int8_gemm_act(*wq, *none).shape == (64, 0)
    torch.cuda.synchronize()
