"""A linear's workspace over one of its operands is refused: the activation's codes would be
written over it before the product reads it.  CPU tensors, as the device is checked last."""
import pytest

import nvfp4_block_scaled_17_b200 as nv
from test_operator_overlaps import F32, I8, U8, BF16, NOT_CUDA, built, fp4_linear, int8_linear, over, z

assert built                           # the fixture that builds the extension module

SHAPES = {int8_linear: {"wq": (I8, 64, 64), "sw": (F32, 64), "bias": (BF16, 64), "x": (BF16, 8, 64),
                        "residual": (BF16, 8, 64)},
          fp4_linear: {"w_packed": (U8, 64, 32), "w_sf": (U8, 512), "bias": (BF16, 64),
                       "x": (BF16, 8, 64), "residual": (BF16, 8, 64)}}
CASES = [(f, name) for f, shapes in SHAPES.items() for name in shapes]


@pytest.mark.parametrize("f,name", CASES)
def test_workspace_over_an_operand(f, name):
    big = z(16384, dtype=U8)
    dtype, *shape = SHAPES[f][name]
    t = over(big, dtype, *shape)
    n = t.numel() * t.element_size()
    for ws in (big, big[:65], big[64 + n - 1:]):         # all of it, its first and last byte
        with pytest.raises(ValueError, match=f"workspace must not overlap {name}"):
            f(**{name: t}, workspace=ws)
    for ws in (big[:64], big[64 + n:]):                  # up to it, and behind it
        with pytest.raises(TypeError, match=NOT_CUDA):
            f(**{name: t}, workspace=ws)


def test_workspace_over_prepared_scales():
    big = z(16384, dtype=U8)
    n = nv.nvfp4_prepared_scale_bytes(64, 64)
    for ws in (big, big[n - 1:]):
        with pytest.raises(ValueError, match="workspace must not overlap w_sf"):
            fp4_linear(w_sf=big[:n], prepared=True, workspace=ws)
    with pytest.raises(TypeError, match=NOT_CUDA):
        fp4_linear(w_sf=big[:n], prepared=True, workspace=big[n:])
