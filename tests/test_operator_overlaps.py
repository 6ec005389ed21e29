"""What the norm and epilogue entry points accept as a scalar, and which overlaps of their
tensors they refuse.  CPU tensors: the checks come before the one for the device, so an accepted
argument ends in that one's TypeError."""
import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv

BF16, F32, U8, I8 = torch.bfloat16, torch.float32, torch.uint8, torch.int8
NOT_CUDA = "must be a CUDA tensor"


@pytest.fixture(scope="module", autouse=True)
def built():
    from nvfp4_block_scaled_17_b200 import _build
    _build.build()


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def over(t, dtype, *shape):
    """A tensor of this type and shape that starts one 64-byte step into t's bytes."""
    n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
    return t.view(-1).view(U8)[64:64 + n].view(dtype).view(*shape)


def int8_norm(**kw):
    a = dict(x=z(8, 64), weight=z(64), eps=1e-6, residual=z(8, 64), residual_out=z(8, 64),
             norm_out=z(8, 64), out=(z(8, 64, dtype=I8), z(8, dtype=F32)))
    return nv.int8_rmsnorm_quantize(**{**a, **kw})


def fp4_norm(**kw):
    a = dict(x=z(8, 64), weight=z(64), gsf=z(1, dtype=F32), eps=1e-6, residual=z(8, 64),
             residual_out=z(8, 64), norm_out=z(8, 64),
             out=(z(8, 32, dtype=U8), z(512, dtype=U8)))
    return nv.nvfp4_rmsnorm_quantize(**{**a, **kw})


def int8_gemm(**kw):
    a = dict(a=z(8, 64, dtype=I8), sa=z(8, dtype=F32), b=z(64, 64, dtype=I8), sb=z(64, dtype=F32),
             bias=z(64), residual=z(8, 64), out=z(8, 64))
    return nv.int8_gemm_act(**{**a, **kw})


def fp4_gemm(**kw):
    a = dict(a=z(8, 32, dtype=U8), sfa=z(512, dtype=U8), b=z(64, 32, dtype=U8),
             sfb=z(512, dtype=U8), alpha=z(1, dtype=F32), bias=z(64), M=8, N=64, K=64,
             residual=z(8, 64), out=z(8, 64))
    return nv.nvfp4_gemm_act(**{**a, **kw})


def int8_linear(**kw):
    a = dict(x=z(8, 64), wq=z(64, 64, dtype=I8), sw=z(64, dtype=F32), bias=z(64),
             residual=z(8, 64), out=z(8, 64), workspace=z(8192, dtype=U8))
    return nv.int8_linear_act(**{**a, **kw})


def fp4_linear(**kw):
    a = dict(x=z(8, 64), w_packed=z(64, 32, dtype=U8), w_sf=z(512, dtype=U8),
             gsf_w=z(1, dtype=F32), N=64, bias=z(64), residual=z(8, 64), out=z(8, 64),
             workspace=z(8192, dtype=U8))
    return nv.nvfp4_linear_act(**{**a, **kw})


@pytest.mark.parametrize("f,names", [(fp4_norm, ["gsf"]), (fp4_gemm, ["alpha"]),
                                     (fp4_linear, ["gsf_w", "gsf_x"])])
def test_scalars_of_any_one_element_shape(f, names):
    for name in names:
        for shape in ((), (1,), (1, 1)):
            with pytest.raises(TypeError, match=NOT_CUDA):
                f(**{name: torch.ones(shape, dtype=F32)})
        with pytest.raises(ValueError, match=f"{name} must be"):
            f(**{name: z(2, dtype=F32)})
    if f is fp4_norm:
        with pytest.raises(TypeError, match=NOT_CUDA):
            f(gsf_w=torch.ones((), dtype=F32), alpha_out=torch.ones((), dtype=F32))


def test_norm_codes_over_other_tensors():
    for name in ("x", "residual", "residual_out", "norm_out"):
        t = z(8, 64)
        with pytest.raises(ValueError, match="codes must not overlap"):
            int8_norm(**{name: t}, out=(over(t, I8, 8, 64), z(8, dtype=F32)))
        with pytest.raises(ValueError, match="scales must not overlap"):
            int8_norm(**{name: t}, out=(z(8, 64, dtype=I8), over(t, F32, 8)))
        with pytest.raises(ValueError, match="packed must not overlap"):
            fp4_norm(**{name: t}, out=(over(t, U8, 8, 32), z(512, dtype=U8)))
        with pytest.raises(ValueError, match="scales must not overlap"):
            fp4_norm(**{name: t}, out=(z(8, 32, dtype=U8), over(t, U8, 512)))
    codes = z(8, 64, dtype=I8)
    with pytest.raises(ValueError, match="scales must not overlap"):
        int8_norm(out=(codes, over(codes, F32, 8)))
    big = z(600, dtype=U8)
    with pytest.raises(ValueError, match="scales must not overlap"):
        fp4_norm(out=(over(big, U8, 8, 32), big[:512]))
    line = z(600)
    with pytest.raises(ValueError, match="codes must not overlap"):
        int8_norm(weight=line[:64], out=(over(line, I8, 8, 64), z(8, dtype=F32)))


@pytest.mark.parametrize("f,operands", [(int8_gemm, ["a", "b", "sa", "sb", "bias"]),
                                        (fp4_gemm, ["a", "b", "sfa", "sfb", "bias"]),
                                        (int8_linear, ["wq", "sw", "bias", "workspace"]),
                                        (fp4_linear, ["w_packed", "w_sf", "bias", "workspace"])])
def test_out_over_operands(f, operands):
    big = z(8192, dtype=U8)
    shapes = {"a": {int8_gemm: (I8, 8, 64), fp4_gemm: (U8, 8, 32)}.get(f),
              "b": {int8_gemm: (I8, 64, 64), fp4_gemm: (U8, 64, 32)}.get(f),
              "sa": (F32, 8), "sb": (F32, 64), "sw": (F32, 64), "bias": (BF16, 64),
              "sfa": (U8, 512), "sfb": (U8, 512), "w_sf": (U8, 512), "wq": (I8, 64, 64),
              "w_packed": (U8, 64, 32), "workspace": (U8, 8192 - 64)}
    out = big[:1024].view(BF16).view(8, 64)
    for name in operands:
        kw = {name: over(big, *shapes[name]), "out": out}
        with pytest.raises(ValueError, match=f"out must not overlap {name}"):
            f(**kw)


@pytest.mark.parametrize("f", [int8_linear, fp4_linear])
def test_workspace_over_inputs(f):
    big = z(8192, dtype=U8)
    t = big[128:128 + 1024].view(BF16).view(8, 64)
    for name in ("x", "residual"):
        with pytest.raises(ValueError, match=f"workspace must not overlap {name}"):
            f(workspace=big, **{name: t})
    # a square linear onto its own input: x is read before anything is written
    x = z(8, 64)
    with pytest.raises(TypeError, match=NOT_CUDA):
        f(x=x, out=x, residual=x)


def test_in_place_residuals_stay_allowed():
    t = z(8, 64)
    for f in (int8_gemm, fp4_gemm, int8_linear, fp4_linear):
        with pytest.raises(TypeError, match=NOT_CUDA):
            f(residual=t, out=t)
    for f in (int8_norm, fp4_norm):
        for name in ("x", "residual"):
            with pytest.raises(TypeError, match=NOT_CUDA):
                f(**{name: t, "residual_out": t})
