"""The products with an epilogue at the end of K: what stands in other rows' scales stays there."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
import plain_ops as P
from test_gpu_epilogue import extras, operands, product, run

pytestmark = pytest.mark.gpu
NAN_SCALE = 0x7F


def scale_at(row, block, K):
    """Byte of a row's 16-value block in the 128x4 layout."""
    groups = (K // 16 + 3) // 4
    return (((row >> 7) * groups + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
            (block & 3))


# every schedule: streaming, clusters, split-K, SM pairs (whole and half tiles); K with one,
# two and three steps in its last stage
SHAPES = [(2, 19200, 576), (2, 19200, 64), (4, 1030, 640), (4, 1030, 192), (300, 520, 2624),
          (300, 520, 576), (300, 520, 704), (2500, 2064, 192), (2500, 2064, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("prepared", [False, True])
def test_nan_scales_stay_in_their_row_and_column(M, N, K, prepared):
    a, sfa, b, sfb, alpha = operands("nvfp4", M, N, K)
    bias, res = extras(M, N, False, True, True)
    clean = run("nvfp4", (a, sfa, b, sfb, alpha), M, N, K, bias, "none", False, res, prepared)
    # the first scales of the row tile after row 72's (and the last row's neighbour below)
    bad_n = [200, N - 1]
    bad_m = [200] if M > 200 else []
    sfa, sfb = sfa.clone(), sfb.clone()
    for block in range(4):
        for n in bad_n:
            sfb[scale_at(n, block, K)] = NAN_SCALE
        for m in bad_m:
            sfa[scale_at(m, block, K)] = NAN_SCALE
    y = run("nvfp4", (a, sfa, b, sfb, alpha), M, N, K, bias, "none", False, res, prepared)
    torch.cuda.synchronize()
    assert nv.last_device_status() == nv.OK
    bad = torch.zeros(M, N, dtype=torch.bool, device=y.device)
    bad[:, bad_n] = True
    bad[bad_m, :] = True
    assert torch.isnan(y[bad]).all()
    assert torch.equal(y[~bad].view(torch.int16), clean[~bad].view(torch.int16))


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M,K", [(1, 1024), (40, 512), (300, 576), (2500, 1088)])
def test_linear_onto_its_own_input(kind, M, K):
    """out is x, and the residual too: x is read, then written."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(K, K, generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    if kind == "int8":
        def call(x, **kw):
            return nv.int8_linear_act(x, *nv.int8_quantize_rows(w), activation="gelu", **kw)
    else:
        def call(x, **kw):
            return nv.nvfp4_linear_act(x, *nv.pack_weight(w), K, activation="gelu", **kw)
    want = call(x, residual=x)
    for _ in range(5):
        live = x.clone()
        call(live, residual=live, out=live)
        torch.cuda.synchronize()
        assert nv.last_device_status() == nv.OK
        assert torch.equal(live.view(torch.int16), want.view(torch.int16))


def test_scalars_without_dimensions():
    M, N, K = 4, 64, 128
    a, sfa, b, sfb, alpha = operands("nvfp4", M, N, K)
    want = nv.nvfp4_gemm_act(a, sfa, b, sfb, alpha.reshape(1), None, M, N, K)
    got = nv.nvfp4_gemm_act(a, sfa, b, sfb, alpha.reshape(()), None, M, N, K)
    x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    gsf = torch.tensor(30.0, device="cuda")
    one = nv.nvfp4_rmsnorm_quantize(x, None, gsf, 1e-6)
    two = nv.nvfp4_rmsnorm_quantize(x, None, gsf.reshape(1), 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


@pytest.mark.parametrize("kind", ["int8", "nvfp4"])
@pytest.mark.parametrize("M,N", [(2500, 2062), (2500, 2061), (2499, 2060), (300, 522), (301, 521),
                                 (129, 2598), (8200, 1033)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_widths_that_tma_cannot_store(kind, M, N, gated, in_place):
    """The columns and rows around y stay as they were, with and without a residual."""
    K, cols = 192, N // 2 if gated else N
    if gated and N % 2:
        N, cols = N + 1, (N + 1) // 2
    ops = operands(kind, M, N, K)
    bias, res = extras(M, N, gated, True, True)
    pad = 64
    whole = torch.full((pad + M * cols + pad,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = whole[pad:pad + M * cols].view(M, cols)
    for r in (res, None):
        if in_place and r is not None:
            y.copy_(r)
        run(kind, ops, M, N, K, bias, "silu", gated, y if in_place and r is not None else r, out=y)
        torch.cuda.synchronize()
        assert nv.last_device_status() == nv.OK
        assert (whole[:pad] == 7.0).all() and (whole[pad + M * cols:] == 7.0).all()
        v, dv = product(kind, ops, M, N, K, bias)
        y64, bound = P.epilogue_64(v, dv, "silu", gated, r)
        P.check(y, y64, bound, f"{kind} {M}x{N} gated={gated} residual={r is not None}")
