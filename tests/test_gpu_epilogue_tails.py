"""The epilogues' activations far from zero: gelu, gelu_tanh and silu end at 0 on the left and
in the value itself on the right, and a NaN stays in its own column."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
import plain_ops as P
from test_gpu_epilogue import operands, product, run

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
INF = float("inf")
SMOOTH = ("gelu", "gelu_tanh", "silu")
# few rows on a long weight, clusters, split-K, SM pairs
SHAPES = [(3, 19200, 128), (3, 512, 256), (90, 512, 2624), (300, 512, 256)]
# bf16 values; the products of these operands stay below 200
FAR = (-3.0e38, -1.0e30, -1.0e20, -1.0e10, -1.0e6, -1.0e4, -1.0e3)


def far_bias(N, values):
    bias = torch.zeros(N, device=DEV)
    for i, v in enumerate(values):
        bias[4 * i + 8] = v
    return bias.to(BF16), [4 * i + 8 for i in range(len(values))]


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", SMOOTH)
def test_left_tail_is_zero(kind, M, N, K, act):
    """At v < -500 the definition is below 1e-200: zero in any of the formats.  (At -inf it
    is no number: -inf * 0.)"""
    ops = operands(kind, M, N, K)
    bias, at = far_bias(N, FAR)
    v, _ = product(kind, ops, M, N, K, bias)
    assert (v[:, at] < -500).all()
    y = run(kind, ops, M, N, K, bias, act, False, None)
    assert (y[:, at] == 0).all()
    # gated, the tail in the gate and a large partner beside it
    bias[[c + 1 for c in at]] = 1.0e30
    y = run(kind, ops, M, N, K, bias, act, True, None)
    assert (y[:, [c // 2 for c in at]] == 0).all()


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", SMOOTH)
def test_right_tail_is_the_value(kind, M, N, K, act):
    ops = operands(kind, M, N, K)
    bias, at = far_bias(N, [INF] + [-v for v in FAR])
    y = run(kind, ops, M, N, K, bias, act, False, None)
    plain = run(kind, ops, M, N, K, bias, "none", False, None)
    assert torch.equal(y[:, at].view(torch.int16), plain[:, at].view(torch.int16))
    assert torch.isinf(y[:, at[0]]).all()


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", SMOOTH)
def test_nan_stays_in_its_column(kind, M, N, K, act):
    """Two values share a reciprocal; a NaN in one leaves the other's bits."""
    ops = operands(kind, M, N, K)
    bias = torch.linspace(-8.0, 8.0, N, device=DEV).to(BF16)
    for gated in (False, True):
        clean = run(kind, ops, M, N, K, bias, act, gated, None)
        broken = bias.clone()
        broken[[20, 41, 66]] = float("nan")
        y = run(kind, ops, M, N, K, broken, act, gated, None)
        cols = [10, 20, 33] if gated else [20, 41, 66]
        bad = torch.zeros(y.shape[1], dtype=torch.bool, device=DEV)
        bad[cols] = True
        assert torch.isnan(y[:, bad]).all()
        assert torch.equal(y[:, ~bad].view(torch.int16), clean[:, ~bad].view(torch.int16))


@pytest.mark.parametrize("act", SMOOTH)
def test_around_the_cut(act):
    """Densely over the left side, against 64 bits, with the stated error."""
    N, K, M = 4096, 128, 2
    a = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    b = torch.zeros(N, K, dtype=torch.int8, device=DEV)
    sa, sb = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    bias = torch.linspace(-60.0, 2.0, N, device=DEV).to(BF16)
    y = nv.int8_gemm_act(a, sa, b, sb, bias, act)
    v, dv = P.int8_product_64(a, sa, b, sb, bias)
    P.check(y, *P.epilogue_64(v, dv, act, False, None), act)
