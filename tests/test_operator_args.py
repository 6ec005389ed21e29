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


BF16, I8, U8, F32 = torch.bfloat16, torch.int8, torch.uint8, torch.float32


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def norms():
    """The two norms as one call each of keyword arguments, with arguments that only a CPU
    tensor makes wrong (the device is checked last)."""
    base = dict(x=z(4, 64), weight=z(64), eps=1e-6, residual=z(4, 64), residual_out=z(4, 64))
    return [(nv.int8_rmsnorm_quantize, dict(base, out=(z(4, 64, dtype=I8), z(4, dtype=F32)))),
            (nv.nvfp4_rmsnorm_quantize,
             dict(base, gsf=z(1, dtype=F32), out=(z(4, 32, dtype=U8), z(512, dtype=U8))))]


def products():
    a, b = z(4, 64, dtype=I8), z(8, 64, dtype=I8)
    p, q, sf = z(4, 32, dtype=U8), z(8, 32, dtype=U8), z(512, dtype=U8)
    one = z(1, dtype=F32)
    base = dict(bias=z(8), activation="silu", residual=z(4, 8), out=z(4, 8))
    ws = z(1 << 16, dtype=U8)
    return [(nv.int8_gemm_act, dict(base, a=a, sa=z(4, dtype=F32), b=b, sb=z(8, dtype=F32))),
            (nv.nvfp4_gemm_act, dict(base, a=p, sfa=sf, b=q, sfb=sf, alpha=one, M=4, N=8, K=64)),
            (nv.int8_linear_act, dict(base, x=z(4, 64), wq=b, sw=z(8, dtype=F32), workspace=ws)),
            (nv.nvfp4_linear_act, dict(base, x=z(4, 64), w_packed=q, w_sf=sf, gsf_w=one, N=8,
                                       workspace=ws))]


def refuses(f, kw, error, match, **change):
    with pytest.raises(error, match=match):
        f(**dict(kw, **change))


def test_norm_tensors():
    for f, kw in norms():
        refuses(f, kw, TypeError, "CUDA")                     # all else is right
        refuses(f, kw, TypeError, "x must be a BFloat16", x=z(4, 64, dtype=torch.float16))
        refuses(f, kw, ValueError, "2-D", x=z(64))
        refuses(f, kw, ValueError, "contiguous", x=z(4, 128)[:, ::2])
        refuses(f, kw, ValueError, "residual must be", residual=z(4, 32))
        refuses(f, kw, TypeError, "residual must be", residual=z(4, 64, dtype=F32))
        refuses(f, kw, ValueError, "weight must be", weight=z(65))
        refuses(f, kw, ValueError, "residual_out must be", residual_out=z(5, 64))
        refuses(f, kw, ValueError, "needs a residual", residual=None)
        refuses(f, kw, ValueError, "norm_out must be", norm_out=z(4, 63))
        refuses(f, kw, TypeError, "weight must be on", weight=z(64).to("meta"))
        refuses(f, kw, TypeError, "eps", eps="small")
        both = z(8, 64)
        refuses(f, kw, ValueError, "residual_out must be x or residual", x=both[:4], residual_out=both[2:6])
        refuses(f, kw, ValueError, "norm_out must not overlap", x=both[:4], norm_out=both[:4])
        refuses(f, kw, ValueError, "norm_out must not overlap", residual_out=both[:4], norm_out=both[3:7])
        refuses(f, kw, TypeError, "CUDA", residual_out=kw["x"])        # in place is right
        refuses(f, kw, TypeError, "CUDA", residual_out=kw["residual"])
        line = z(5, 64)
        refuses(f, kw, ValueError, "weight must not overlap", weight=line[4], residual_out=line[1:])
    (f8, k8), (f4, k4) = norms()
    refuses(f8, k8, ValueError, "codes", out=(z(4, 63, dtype=I8), z(4, dtype=F32)))
    refuses(f8, k8, ValueError, "scales", out=(z(4, 64, dtype=I8), z(5, dtype=F32)))
    refuses(f4, k4, ValueError, "packed", out=(z(4, 64, dtype=U8), z(512, dtype=U8)))
    refuses(f4, k4, ValueError, "scales", out=(z(4, 32, dtype=U8), z(511, dtype=U8)))
    refuses(f4, k4, ValueError, "gsf must be", gsf=z(2, dtype=F32))
    refuses(f4, k4, TypeError, "gsf must be a tensor", gsf=1.0)
    refuses(f4, k4, TypeError, "alpha_out", alpha_out=z(1))


def test_product_tensors():
    for f, kw in products():
        refuses(f, kw, TypeError, "CUDA")
        refuses(f, kw, ValueError, "activation", activation="swish")
        refuses(f, kw, ValueError, "bias must be", bias=z(9))
        refuses(f, kw, TypeError, "bias must be", bias=z(8, dtype=F32))
        refuses(f, kw, ValueError, "out must be", out=z(4, 7))
        refuses(f, kw, ValueError, "out must be", gated=True)          # needs N / 2 columns
        refuses(f, kw, ValueError, "residual must be", residual=z(4, 16)[:, ::2])
        refuses(f, kw, TypeError, "residual must be on", residual=z(4, 8).to("meta"))
        both = z(8, 8)
        refuses(f, kw, ValueError, "residual must be out", residual=both[:4], out=both[1:5])
        refuses(f, kw, TypeError, "CUDA", residual=kw["out"])          # in place is right
        refuses(f, kw, TypeError, "CUDA", gated=True, out=z(4, 4), residual=None)
    (g8, a8), (g4, a4), (l8, b8), (l4, b4) = products()
    refuses(g8, a8, ValueError, "even", gated=True, b=z(9, 64, dtype=I8))
    refuses(g8, a8, ValueError, "b must be", b=z(8, 32, dtype=I8))
    refuses(g8, a8, ValueError, "sa must be", sa=z(5, dtype=F32))
    refuses(g8, a8, TypeError, "a must be", a=z(4, 64, dtype=U8))
    refuses(g4, a4, ValueError, "a must be", a=z(4, 31, dtype=U8))
    refuses(g4, a4, ValueError, "sfb must be", sfb=z(511, dtype=U8))
    refuses(g4, a4, ValueError, "sfb must be", prepared=True)          # prepared blocks are longer
    refuses(g4, a4, ValueError, "alpha must be", alpha=z(2, dtype=F32))
    refuses(l8, b8, TypeError, "workspace", workspace=z(64))
    refuses(l4, b4, ValueError, "w_packed", w_packed=z(8, 31, dtype=U8))
    refuses(l4, b4, ValueError, "gsf_x must be", gsf_x=z(0, dtype=F32))


def test_extension_module():
    calls = nv._calls()
    assert all(hasattr(calls, n) for n in nv._BOUND[:6])
    with pytest.raises(TypeError):
        calls.int8_rmsnorm_quantize(1, 2)                              # wrong number of arguments
    with pytest.raises(TypeError, match="x must be a tensor"):
        calls.int8_rmsnorm_quantize(*([None] * 9))


def test_interleave_gate_up():
    g, u = torch.arange(6.0).view(3, 2), torch.arange(6.0).view(3, 2) + 100
    w = nv.interleave_gate_up(g, u)
    assert torch.equal(w[0::2], g) and torch.equal(w[1::2], u)
    assert torch.equal(nv.interleave_gate_up(g[:, 0], u[:, 0])[1::2], u[:, 0])
    with pytest.raises(ValueError):
        nv.interleave_gate_up(g, u[:2])
