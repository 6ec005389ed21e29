"""Device scalars (global scales, alpha) under an output or a workspace are refused: a kernel
would overwrite them while its other blocks still read them.  CPU tensors, as the device is
checked last."""
import pytest

from test_operator_overlaps import (F32, NOT_CUDA, U8, built, fp4_gemm, fp4_linear, fp4_norm, z)

assert built                           # the fixture that builds the extension module


def scalar_in(t, at=64):
    """One float32 inside t's bytes."""
    return t.view(-1).view(U8)[at:at + 4].view(F32)


@pytest.mark.parametrize("name", ["gsf", "gsf_w"])
@pytest.mark.parametrize("output", ["residual_out", "norm_out", "packed", "scales"])
def test_norm_scalars_under_an_output(name, output):
    t = {"residual_out": z(8, 64), "norm_out": z(8, 64), "packed": z(8, 32, dtype=U8),
         "scales": z(512, dtype=U8)}[output]
    kw = {output: t} if output.endswith("_out") else {}
    kw["out"] = (t if output == "packed" else z(8, 32, dtype=U8),
                 t if output == "scales" else z(512, dtype=U8))
    kw.update(gsf_w=z(1, dtype=F32), alpha_out=z(1, dtype=F32))
    with pytest.raises(ValueError, match=f"{name} must not overlap"):
        fp4_norm(**{**kw, name: scalar_in(t)})
    with pytest.raises(TypeError, match=NOT_CUDA):
        fp4_norm(**kw)


@pytest.mark.parametrize("other", ["gsf", "gsf_w", "x", "residual", "weight", "residual_out",
                                   "norm_out", "packed", "scales"])
def test_alpha_out_over_another_tensor(other):
    t = {"gsf": z(1, dtype=F32), "gsf_w": z(1, dtype=F32), "weight": z(64),
         "packed": z(8, 32, dtype=U8), "scales": z(512, dtype=U8)}.get(other)
    t = z(8, 64) if t is None else t
    kw = dict(gsf_w=z(1, dtype=F32))
    if other in ("packed", "scales"):
        kw["out"] = (t if other == "packed" else z(8, 32, dtype=U8),
                     t if other == "scales" else z(512, dtype=U8))
    else:
        kw[other] = t
    alpha = t if t.numel() == 1 else scalar_in(t)
    with pytest.raises(ValueError, match="alpha_out must not overlap"):
        fp4_norm(**kw, alpha_out=alpha)


def test_products_over_their_scalars():
    out = z(8, 64)
    with pytest.raises(ValueError, match="out must not overlap alpha"):
        fp4_gemm(alpha=scalar_in(out), out=out)
    ws = z(8192, dtype=U8)
    for name in ("gsf_w", "gsf_x"):
        with pytest.raises(ValueError, match=f"out must not overlap {name}"):
            fp4_linear(**{name: scalar_in(out)}, out=out)
        with pytest.raises(ValueError, match=f"workspace must not overlap {name}"):
            fp4_linear(**{name: scalar_in(ws)}, workspace=ws)


def test_scalars_that_share_their_memory_as_inputs_are_right():
    one = z(1, dtype=F32)
    with pytest.raises(TypeError, match=NOT_CUDA):
        fp4_linear(gsf_w=one, gsf_x=one)
    with pytest.raises(TypeError, match=NOT_CUDA):
        fp4_norm(gsf=one, gsf_w=one, alpha_out=z(1, dtype=F32))
    line = z(4, dtype=F32)                                 # neighbours, as a program keeps them
    with pytest.raises(TypeError, match=NOT_CUDA):
        fp4_norm(gsf=line[0:1], gsf_w=line[1:2], alpha_out=line[2:3])
