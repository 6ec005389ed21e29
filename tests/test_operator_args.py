"""Refusals of the norm and epilogue entry points: through the C ABI with addresses that are
never dereferenced, and through the binding with CPU tensors.  Nothing runs on a device."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv

A = ctypes.c_void_p(1 << 20)
MIS = ctypes.c_void_p((1 << 20) + 4)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def L():
    from nvfp4_block_scaled_17_b200 import _build
    _build.build()
    return nv.lib()


def int8_norm(L, x=A, r=A, w=A, eps=1e-6, rows=4, K=64, q=A, s=A, h=A, n=None):
    return L.int8_rmsnorm_quantize(x, r, w, eps, rows, K, q, s, h, n, None)


def nvfp4_norm(L, x=A, r=A, w=A, eps=1e-6, rows=4, K=64, gsf=A, p=A, sf=A, gw=None, al=None, h=A,
               n=None):
    return L.nvfp4_rmsnorm_quantize(x, r, w, eps, rows, K, gsf, p, sf, gw, al, h, n, None)


@pytest.mark.parametrize("f", [int8_norm, nvfp4_norm])
def test_norm_arguments(L, f):
    assert f(L, x=None) == nv.ERR_INVALID_ARG
    assert f(L, rows=-1) == nv.ERR_INVALID_ARG
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert f(L, eps=eps) == nv.ERR_INVALID_ARG
    assert f(L, r=None) == nv.ERR_INVALID_ARG              # residual_out without a residual
    for K in (0, -16, 24, 65552):
        assert f(L, K=K) == nv.ERR_SHAPE
    for name in ("x", "r", "w", "h", "n"):
        assert f(L, **{name: MIS}) == nv.ERR_ALIGN


def test_norm_outputs(L):
    assert int8_norm(L, q=None) == nv.ERR_INVALID_ARG
    assert int8_norm(L, s=None) == nv.ERR_INVALID_ARG
    assert int8_norm(L, q=MIS) == nv.ERR_ALIGN
    assert int8_norm(L, s=ODD) == nv.ERR_ALIGN
    for name in ("gsf", "p", "sf"):
        assert nvfp4_norm(L, **{name: None}) == nv.ERR_INVALID_ARG
    assert nvfp4_norm(L, gw=A) == nv.ERR_INVALID_ARG       # gsf_w alone
    assert nvfp4_norm(L, al=A) == nv.ERR_INVALID_ARG
    assert nvfp4_norm(L, p=MIS) == nv.ERR_ALIGN
    assert nvfp4_norm(L, sf=MIS) == nv.ERR_ALIGN
    assert nvfp4_norm(L, gsf=ODD) == nv.ERR_ALIGN
    assert nvfp4_norm(L, gw=ODD, al=A) == nv.ERR_ALIGN


def int8_gemm(L, a=A, sa=A, b=A, sb=A, bias=A, act=4, res=A, y=A, M=4, N=8, K=64):
    return L.int8_gemm_act(a, sa, b, sb, bias, act, res, y, M, N, K, None)


def nvfp4_gemm(L, a=A, sa=A, b=A, sb=A, bias=A, act=4, res=A, y=A, M=4, N=8, K=64, prep=0, al=A):
    return L.nvfp4_gemm_act(a, sa, b, sb, prep, al, bias, act, res, y, M, N, K, None)


def int8_linear(L, a=A, b=A, sb=A, bias=A, act=4, res=A, y=A, M=4, N=8, K=64, ws=A, nws=1 << 20):
    return L.int8_linear_act(a, M, K, b, sb, N, bias, act, res, ws, nws, y, None)


def nvfp4_linear(L, a=A, b=A, sb=A, bias=A, act=4, res=A, y=A, M=4, N=8, K=64, prep=0, al=A, g=0,
                 ws=A, nws=1 << 20):
    return L.nvfp4_linear_act(a, M, K, b, sb, prep, al, N, bias, None, g, act, res, ws, nws, y, None)


@pytest.mark.parametrize("f", [int8_gemm, nvfp4_gemm, int8_linear, nvfp4_linear])
def test_product_arguments(L, f):
    for name in ("a", "b", "sb", "y"):
        assert f(L, **{name: None}) == nv.ERR_INVALID_ARG
        assert f(L, **{name: MIS}) == nv.ERR_ALIGN
    assert f(L, bias=MIS) == nv.ERR_ALIGN
    assert f(L, res=MIS) == nv.ERR_ALIGN
    for act in (-1, 5, 15, 21, 32, 36, 1 << 20):
        assert f(L, act=act) == nv.ERR_INVALID_ARG
    for act in (16, 17, 20):
        assert f(L, act=act, N=9) == nv.ERR_SHAPE          # gated, N odd
    assert f(L, M=-1) == nv.ERR_INVALID_ARG
    assert f(L, N=1 << 31) == nv.ERR_INVALID_ARG
    for K in (0, 48, 1 << 31):
        assert f(L, K=K) == nv.ERR_SHAPE


def test_product_extras(L):
    assert int8_gemm(L, sa=MIS) == nv.ERR_ALIGN
    assert int8_gemm(L, K=131072) == nv.ERR_SHAPE          # the sum could pass 32 bits
    assert int8_linear(L, K=131072, nws=1 << 30) == nv.ERR_SHAPE
    assert nvfp4_gemm(L, sa=None) == nv.ERR_INVALID_ARG
    for f in (nvfp4_gemm, nvfp4_linear):
        assert f(L, prep=2) == nv.ERR_INVALID_ARG
        assert f(L, al=None) == nv.ERR_INVALID_ARG
        assert f(L, al=ODD) == nv.ERR_ALIGN
    for f in (int8_linear, nvfp4_linear):
        assert f(L, ws=None) == nv.ERR_WORKSPACE
        assert f(L, nws=16) == nv.ERR_WORKSPACE
        assert f(L, ws=ctypes.c_void_p((1 << 20) + 16)) == nv.ERR_ALIGN
    assert nvfp4_linear(L, g=48) == nv.ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 64, dtype=torch.int8)
    s = torch.zeros(4)
    u = torch.zeros(4, 32, dtype=torch.uint8)
    for call in (lambda: nv.int8_rmsnorm_quantize(x, None, 1e-6),
                 lambda: nv.nvfp4_rmsnorm_quantize(x, None, s[:1], 1e-6),
                 lambda: nv.int8_gemm_act(q, s, q, s),
                 lambda: nv.nvfp4_gemm_act(u, u, u, u, s[:1], None, 4, 4, 64),
                 lambda: nv.int8_linear_act(x, q, s),
                 lambda: nv.nvfp4_linear_act(x, u, u, s[:1], 4)):
        with pytest.raises(TypeError):
            call()


class FakeTensor:
    """What the binding's checks read of a tensor, at a made-up address."""
    is_cuda = True

    def __init__(self, shape, dtype, ptr, device="cuda:0", contiguous=True):
        self.shape, self.dtype, self.ptr = torch.Size(shape), dtype, ptr
        self.device, self.c = torch.device(device), contiguous

    def is_contiguous(self):
        return self.c

    def data_ptr(self):
        return self.ptr

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()


BF16 = torch.bfloat16


def test_argument_checks(monkeypatch):
    dev = torch.device("cuda:0")
    t = FakeTensor((4, 64), BF16, 4096)
    assert nv._need(t, "t", (4, 64), BF16, dev) == 4096
    assert nv._need(None, "t", (4, 64), BF16, dev) is None
    for bad in (FakeTensor((4, 64), torch.float16, 0), FakeTensor((4, 64), BF16, 0, "cuda:1")):
        with pytest.raises(TypeError):
            nv._need(bad, "t", (4, 64), BF16, dev)
    for bad in (FakeTensor((4, 63), BF16, 0), FakeTensor((4, 64), BF16, 0, contiguous=False)):
        with pytest.raises(ValueError):
            nv._need(bad, "t", (4, 64), BF16, dev)
    with pytest.raises(ValueError):
        nv._need_bytes(FakeTensor((15,), torch.uint8, 0), "t", 16, dev)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        nv._here(t, "t")


def test_overlaps_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = FakeTensor((4, 64), BF16, 4096)
    r = FakeTensor((4, 64), BF16, 8192)
    half = FakeTensor((4, 64), BF16, 4096 + 256)
    with pytest.raises(ValueError, match="residual_out"):
        nv._norm_inputs(x, None, r, half, None)
    with pytest.raises(ValueError, match="residual_out"):
        nv._norm_inputs(x, None, None, r, None)
    with pytest.raises(ValueError, match="norm_out"):
        nv._norm_inputs(x, None, r, r, x)
    nv._norm_inputs(x, None, r, r, None)                   # in place is fine
    y = FakeTensor((4, 8), BF16, 4096)
    near = FakeTensor((4, 8), BF16, 4096 + 16)
    with pytest.raises(ValueError, match="residual"):
        nv._epilogue("silu", False, near, None, y, 4, 8, x.device)
    nv._epilogue("silu", False, y, None, y, 4, 8, x.device)
    with pytest.raises(ValueError, match="even"):
        nv._epilogue("silu", True, None, None, None, 4, 9, x.device)
    with pytest.raises(ValueError, match="activation"):
        nv._epilogue("swish", False, None, None, y, 4, 8, x.device)


def test_interleave_gate_up():
    g, u = torch.arange(6.0).view(3, 2), torch.arange(6.0).view(3, 2) + 100
    w = nv.interleave_gate_up(g, u)
    assert torch.equal(w[0::2], g) and torch.equal(w[1::2], u)
    assert torch.equal(nv.interleave_gate_up(g[:, 0], u[:, 0])[1::2], u[:, 0])
    with pytest.raises(ValueError):
        nv.interleave_gate_up(g, u[:2])
