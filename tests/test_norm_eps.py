"""The smallest eps of the norms: below 2^-255 the root's reciprocal would pass fp32's range, and
a row of zeros would give 0 * inf."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from test_operator_args import L, int8_norm, nvfp4_norm

assert L                               # the fixture that loads the library


@pytest.mark.parametrize("f", [int8_norm, nvfp4_norm])
def test_eps_that_fp32_cannot_hold(L, f):
    for eps in (1e-80, 1e-300, 5e-324, 2.0 ** -256):
        assert f(L, eps=eps) == nv.ERR_INVALID_ARG
    for eps in (2.0 ** -255, 1e-76, 1e-45, 1e-6, 1e300):     # right; K is not
        assert f(L, eps=eps, K=24) == nv.ERR_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("K", [80, 2048])
def test_rows_of_zeros_at_the_smallest_eps(K):
    x = torch.zeros(3, K, device="cuda").to(torch.bfloat16)
    x[1] = 9.2e-41                                           # the smallest bf16 value
    n = torch.empty_like(x)
    for eps in (2.0 ** -255, 1e-45):
        q, s, _ = nv.int8_rmsnorm_quantize(x, None, eps, norm_out=n)
        p, sf, _ = nv.nvfp4_rmsnorm_quantize(x, None, torch.ones(1, device="cuda"), eps)
        torch.cuda.synchronize()
        for row in (0, 2):
            assert (n[row] == 0).all() and (q[row] == 0).all() and s[row] == 0
            assert (p[row] == 0).all()
        assert torch.isfinite(n[1]).all() and (n[1] > 0).all() and (q[1] == 127).all()
