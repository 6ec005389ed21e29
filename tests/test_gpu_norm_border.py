"""Rows of 33 to 64 units around the number of rows where the norms change their layout."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from test_gpu_norm_nonfinite import EPS, inputs, same_bits
from plain_ops import norm_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [2368, 2399, 2400, 2401, 4095, 4096])
@pytest.mark.parametrize("K", [528, 1024])
def test_both_sides_of_the_border(R, K):
    x, r, w = inputs(R, K)
    n = torch.empty_like(x)
    q, s, h = nv.int8_rmsnorm_quantize(x, w, EPS, residual=r, norm_out=n)
    gsf = torch.tensor([77.7], device="cuda")
    p, sf, h2 = nv.nvfp4_rmsnorm_quantize(x, w, gsf, EPS, residual=r)
    q2, s2 = nv.int8_quantize_rows(n)
    p2, sf2, _ = nv.nvfp4_quantize(n, 0, gsf)
    torch.cuda.synchronize()
    h_ref, n_ref = norm_rows(x, r, w, EPS)
    assert same_bits(h, h_ref) and same_bits(h2, h_ref) and same_bits(n, n_ref)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(p, p2) and torch.equal(sf, sf2)
