"""int8_rmsnorm_quantize and nvfp4_rmsnorm_quantize on the GPU: codes, scales, h and n bit for
bit against a plain implementation (sum and root in 64 bits) followed by the oracle's
quantizers, and n against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from nvfp4_block_scaled_17_b200 import workloads as W
from gpu_util import to_np
from plain_ops import norm_rows, norm_rows_64

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
SHAPES = [(1, 16), (1, 5120), (3, 48), (37, 80), (129, 512), (5, 528), (64, 1024), (7, 1040),
          (33, 2048), (9, 2064), (300, 5120), (700, 496), (6, 544), (2, 16384), (3, 16400), (2, 25600), (1, 32784),
          (2, 65536)]


def inputs(R, K, residual=True, weight=True, seed=0):
    g = W._gen(seed + 31 * R + K, "cpu")
    x = W.with_outliers((R, K), 0.01, 20.0, g, "cpu")
    x = (x.float() * torch.exp(torch.randn(R, 1, generator=g))).to(torch.bfloat16)
    r = W.normal((R, K), 2.0, g, "cpu").to(torch.bfloat16) if residual else None
    w = (1.0 + W.normal((K,), 0.3, g, "cpu")).to(torch.bfloat16) if weight else None
    return x, r, w


def on(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def same(a, b):
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))


def check_n(n, h, w):
    """n against 64 bits: rstd and the two products are three roundings of 2^-24, the last
    one half a bf16 step (2^-8) more."""
    n64 = norm_rows_64(h, w, EPS)
    bound = n64.abs() * (3 * 2.0 ** -24 + 2.0 ** -8) * 1.001 + 2.0 ** -134
    assert ((n.cpu().double() - n64).abs() <= bound).all()


@pytest.mark.parametrize("R,K", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_int8(oracle, R, K, residual):
    x, r, w = inputs(R, K, residual)
    if R > 2:
        x[1] = 0.0
        if r is not None:
            r[1] = 0.0                                    # a row of zeros
    dx, dr, dw = on(x, r, w)
    n_out = torch.empty_like(dx)
    q, s, h = nv.int8_rmsnorm_quantize(dx, dw, EPS, residual=dr, norm_out=n_out)
    torch.cuda.synchronize()
    h_ref, n_ref = norm_rows(x, r, w, EPS)
    if residual:
        assert same(h, h_ref)
    else:
        assert h is None
    assert same(n_out, n_ref)
    check_n(n_out, h_ref, w)
    oq, os_ = oracle.int8_quantize_rows(W.to_u16(n_ref))
    assert np.array_equal(to_np(s), os_[:R])
    assert np.array_equal(to_np(q), oq)


@pytest.mark.parametrize("R,K", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_nvfp4(oracle, R, K, residual):
    x, r, w = inputs(R, K, residual, seed=5)
    if R > 2:
        x[R - 1] = 0.0
        if r is not None:
            r[R - 1] = 0.0
    dx, dr, dw = on(x, r, w)
    gsf = torch.tensor([2688.0 / 9.7], device=DEV)        # some values saturate
    gw = torch.tensor([123.4], device=DEV)
    alpha = torch.zeros(1, device=DEV)
    out = (torch.full((R, K // 2), 0xAA, dtype=torch.uint8, device=DEV),
           torch.full((nv.nvfp4_scale_bytes(R, K),), 0xAA, dtype=torch.uint8, device=DEV))
    n_out = torch.empty_like(dx)
    p, sf, h = nv.nvfp4_rmsnorm_quantize(dx, dw, gsf, EPS, residual=dr, out=out, norm_out=n_out,
                                         gsf_w=gw, alpha_out=alpha)
    torch.cuda.synchronize()
    h_ref, n_ref = norm_rows(x, r, w, EPS)
    assert same(n_out, n_ref)
    assert h is None if r is None else same(h, h_ref)
    op, osf, _ = oracle.quantize(W.to_u16(n_ref), float(gsf.item()))
    assert np.array_equal(to_np(p), op)
    assert np.array_equal(to_np(sf), osf)                 # padding rows and columns included
    assert float(alpha) == oracle.alpha(float(gsf), float(gw))


@pytest.mark.parametrize("K", [1024, 5120])
def test_many_rows(oracle, K):
    """More rows than are resident at once: every row group strides over several rows."""
    R = 5000
    x, r, w = inputs(R, K, seed=2)
    dx, dr, dw = on(x, r, w)
    q, s, h = nv.int8_rmsnorm_quantize(dx, dw, EPS, residual=dr)
    gsf = torch.tensor([100.3], device=DEV)
    p, sf, h2 = nv.nvfp4_rmsnorm_quantize(dx, dw, gsf, EPS, residual=dr)
    torch.cuda.synchronize()
    h_ref, n_ref = norm_rows(x, r, w, EPS)
    oq, os_ = oracle.int8_quantize_rows(W.to_u16(n_ref))
    assert same(h, h_ref) and same(h2, h_ref)
    assert np.array_equal(to_np(q), oq) and np.array_equal(to_np(s), os_[:R])
    op, osf, _ = oracle.quantize(W.to_u16(n_ref), float(gsf.item()))
    assert np.array_equal(to_np(p), op) and np.array_equal(to_np(sf), osf)


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e30])
def test_range(oracle, scale):
    """Squares far outside fp32's range on both sides."""
    x, r, w = inputs(9, 1040, seed=3)
    x = (x.float() * scale).to(torch.bfloat16)
    r = (r.float() * scale).to(torch.bfloat16)
    n_out = torch.empty(9, 1040, dtype=torch.bfloat16, device=DEV)
    q, s, h = nv.int8_rmsnorm_quantize(*on(x, w), EPS, residual=r.to(DEV), norm_out=n_out)
    torch.cuda.synchronize()
    h_ref, n_ref = norm_rows(x, r, w, EPS)
    assert same(h, h_ref) and same(n_out, n_ref)
    oq, os_ = oracle.int8_quantize_rows(W.to_u16(n_ref))
    assert np.array_equal(to_np(q), oq) and np.array_equal(to_np(s), os_[:9])


@pytest.mark.parametrize("K", [80, 2048, 5120, 16400])
def test_in_place_and_no_weight(K):
    x, r, _ = on(*inputs(11, K, seed=4))
    want = nv.int8_rmsnorm_quantize(x, None, EPS, residual=r)
    ones = nv.int8_rmsnorm_quantize(x, torch.ones(K, dtype=torch.bfloat16, device=DEV), EPS,
                                    residual=r)
    for into in ("x", "residual"):
        xx, rr = x.clone(), r.clone()
        got = nv.int8_rmsnorm_quantize(xx, None, EPS, residual=rr,
                                       residual_out=xx if into == "x" else rr)
        assert got[2] is (xx if into == "x" else rr)
        for a, b, c in zip(got, want, ones):
            assert torch.equal(a, b) and torch.equal(c, b)


def test_equals_the_separate_passes():
    x, r, w = on(*inputs(130, 5120, seed=6))
    n = torch.empty_like(x)
    gsf = torch.tensor([77.7], device=DEV)
    q, s, _ = nv.int8_rmsnorm_quantize(x, w, EPS, residual=r, norm_out=n)
    p, sf, _ = nv.nvfp4_rmsnorm_quantize(x, w, gsf, EPS, residual=r)
    q2, s2 = nv.int8_quantize_rows(n)
    p2, sf2, _ = nv.nvfp4_quantize(n, 0, gsf)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert torch.equal(p, p2) and torch.equal(sf, sf2)


def test_rows_behind_the_last_are_left():
    x, r, w = on(*inputs(5, 1040, seed=7))
    q = torch.full((8, 1040), 99, dtype=torch.int8, device=DEV)
    s = torch.full((8,), 7.0, device=DEV)
    h = torch.full((8, 1040), 3.0, dtype=torch.bfloat16, device=DEV)
    nv.int8_rmsnorm_quantize(x, w, EPS, residual=r, out=(q[:5], s[:5]), residual_out=h[:5])
    assert (q[5:] == 99).all() and (s[5:] == 7.0).all() and (h[5:] == 3.0).all()


def test_no_rows_and_other_stream():
    x, r, w = on(*inputs(64, 1024, seed=8))
    q, s, h = nv.int8_rmsnorm_quantize(x[:0], w, EPS, residual=r[:0])
    assert q.shape == (0, 1024) and s.shape == (0,) and h.shape == (0, 1024)
    want = nv.int8_rmsnorm_quantize(x, w, EPS, residual=r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = nv.int8_rmsnorm_quantize(x, w, EPS, residual=r)
    explicit = nv.int8_rmsnorm_quantize(x, w, EPS, residual=r, stream=side)
    side.synchronize()
    for a, b, c in zip(got, want, explicit):
        assert torch.equal(a, b) and torch.equal(c, b)


def test_refusals_with_cuda_tensors():
    x, r, w = on(*inputs(4, 64, seed=9))
    with pytest.raises(TypeError, match="must be on"):
        nv.int8_rmsnorm_quantize(x, w.cpu(), EPS, residual=r)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.int8_rmsnorm_quantize(x, w, 0.0, residual=r)
    assert e.value.status == nv.ERR_INVALID_ARG
    with pytest.raises(nv.NVFP4Error) as e:
        nv.int8_rmsnorm_quantize(x[:, :24].contiguous(), w[:24], EPS)
    assert e.value.status == nv.ERR_SHAPE
    big = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, 64)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.int8_rmsnorm_quantize(big, w, EPS)
    assert e.value.status == nv.ERR_ALIGN
