"""The norms' codes where n is not finite: NaN and infinities in x, the residual and the weight,
and values that overflow.  They equal those of the separate passes on the same n."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from nvfp4_block_scaled_17_b200 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
NAN, INF = float("nan"), float("inf")


def inputs(R, K):
    g = W._gen(R + K, "cpu")
    x = W.with_outliers((R, K), 0.01, 20.0, g, "cpu")
    r = W.normal((R, K), 2.0, g, "cpu").to(torch.bfloat16)
    w = (1.0 + W.normal((K,), 0.3, g, "cpu")).to(torch.bfloat16)
    return x.to(DEV), r.to(DEV), w.to(DEV)


def same_bits(a, b):
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(kind), b.view(kind))


def check(x, r, w):
    n = torch.empty_like(x)
    q, s, _ = nv.int8_rmsnorm_quantize(x, w, EPS, residual=r, norm_out=n)
    gsf = torch.tensor([2688.0 / 9.7], device=DEV)
    p, sf, _ = nv.nvfp4_rmsnorm_quantize(x, w, gsf, EPS, residual=r)
    q2, s2 = nv.int8_quantize_rows(n)
    p2, sf2, _ = nv.nvfp4_quantize(n, 0, gsf)
    torch.cuda.synchronize()
    assert not torch.isfinite(n).all()                   # the case is one
    assert same_bits(s, s2) and same_bits(q, q2)
    assert same_bits(sf, sf2) and same_bits(p, p2)
    return n, q


# a warp per row, one and two units a lane; a block per row, one and two units a thread
SHAPES = [(9, 80), (9, 512), (4100, 1024), (9, 1040), (9, 16400)]


@pytest.mark.parametrize("R,K", SHAPES)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_in_the_weight(R, K, value):
    """The row's scale comes from its values that are no NaN; a NaN has the code 0."""
    x, r, w = inputs(R, K)
    x[:, 5], r[:, 5] = 3.0, 1.0                          # times an infinity: an infinity
    w[5] = value
    n, q = check(x, r, w)
    if value != value:
        assert torch.isnan(n[:, 5]).all() and torch.isfinite(n[:, 6:]).all()
        assert (q[:, 5] == 0).all() and (q.abs().amax(1) == 127).all()


@pytest.mark.parametrize("R,K", SHAPES)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("where", ["x", "residual"])
def test_in_a_row(R, K, value, where):
    x, r, w = inputs(R, K)
    clean = nv.int8_rmsnorm_quantize(x, w, EPS, residual=r)[0]
    (x if where == "x" else r)[3, K - 2] = value
    _, q = check(x, r, w)
    others = [i for i in range(R) if i != 3]
    assert torch.equal(q[others], clean[others])         # the other rows as they were


@pytest.mark.parametrize("R,K", SHAPES)
def test_overflow(R, K):
    """Finite inputs whose sum, or whose product with the weight, has no finite bf16 value."""
    x, r, w = inputs(R, K)
    x[1, 7], r[1, 7] = 3.0e38, 3.0e38
    w[K - 1] = 3.3e38
    x[2], r[2] = 0.0, 0.0
    x[2, K - 1] = 4.0
    check(x, r, w)
