"""The largest numbers of rows and columns of the products with an epilogue.  The C ABI with
addresses that are never dereferenced; nothing runs on a device."""
import pytest

import nvfp4_block_scaled_17_b200 as nv
from test_operator_args import L, int8_gemm, int8_linear, nvfp4_gemm, nvfp4_linear

assert L                               # the fixture that loads the library


@pytest.mark.parametrize("f", [int8_gemm, nvfp4_gemm, int8_linear, nvfp4_linear])
@pytest.mark.parametrize("name", ["M", "N"])
def test_rows_and_columns_near_the_end_of_32_bits(L, f, name):
    """The last tile's columns are counted in 32 bits past N: the largest size leaves room."""
    for size in (2 ** 31 - 511, 2 ** 31 - 2, 2 ** 31, 2 ** 40):
        assert f(L, **{name: size}) == nv.ERR_INVALID_ARG
    assert f(L, **{name: 2 ** 31 - 512}, K=48) == nv.ERR_SHAPE       # right; K is not
