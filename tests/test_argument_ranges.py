"""Integers at the ends of their range: what does not fit is refused, not cut off."""
import pytest

from test_operator_overlaps import NOT_CUDA, U8, built, fp4_gemm, fp4_linear, z

assert built                           # the fixture that builds the extension module


@pytest.mark.parametrize("value", [2 ** 32, 2 ** 32 + 1, -2 ** 32, 2 ** 31, 2 ** 62])
def test_integers_beyond_32_bits(value):
    big = z(1 << 16, dtype=U8)
    with pytest.raises(ValueError, match="prepared is out of range"):
        fp4_gemm(prepared=value, sfb=big)
    with pytest.raises(ValueError, match="prepared is out of range"):
        fp4_linear(prepared=value, w_sf=big)
    with pytest.raises(ValueError, match="rotate_group is out of range"):
        fp4_linear(rotate_group=value + 16)
    for kw in (dict(prepared=False), dict(prepared=1, sfb=big)):
        with pytest.raises(TypeError, match=NOT_CUDA):
            fp4_gemm(**kw)
