"""Calls of no rows or no columns through the C ABI: a tensor without elements has no address (an
empty PyTorch tensor's is 0), and only the others' are asked for.  K is wrong in each call, so
that what passes the addresses ends in NVFP4_ERR_SHAPE and nothing runs on a device."""
import pytest

import nvfp4_block_scaled_17_b200 as nv
from test_abi import A, L, S

assert L                               # the fixture that loads the library
SHAPE, INVALID = nv.ERR_SHAPE, nv.ERR_INVALID_ARG


def test_quantizers_of_no_rows(L):
    assert L.hadamard_rotate(None, None, 0, 24, 16, S) == SHAPE
    assert L.nvfp4_quantize(None, 0, 24, 0, A, A, None, None, None, None, A, 4096, S) == SHAPE
    assert L.int8_quantize_rows(None, 0, 24, None, None, S) == SHAPE
    assert L.nvfp4_dequantize(None, None, A, 0, 24, None, S) == SHAPE
    assert L.nvfp4_prepare_weight_scales(None, 0, 24, None, S) == SHAPE
    assert L.int8_rmsnorm_quantize(None, None, None, 1e-6, 0, 24, None, None, None, None, S) == SHAPE
    assert L.nvfp4_rmsnorm_quantize(None, None, None, 1e-6, 0, 24, A, None, None, None, None, None,
                                    None, S) == SHAPE
    # what a call of no rows still needs, and one of a row
    assert L.nvfp4_quantize(None, 0, 24, 0, None, None, None, None, None, None, A, 4096, S) == INVALID
    assert L.nvfp4_dequantize(None, None, None, 0, 24, None, S) == INVALID
    assert L.int8_quantize_rows(None, 1, 24, A, A, S) == INVALID
    assert L.int8_quantize_rows(A, 1, 24, None, A, S) == INVALID
    assert L.int8_quantize_rows(A, 1, 24, A, None, S) == INVALID
    assert L.int8_quantize_rows(None, -1, 24, None, None, S) == INVALID


PRODUCTS = {
    "nvfp4_gemm": lambda L, a, b, y, M, N: L.nvfp4_gemm(a, a, b, b, A, None, y, M, N, 24, S),
    "nvfp4_gemm_prepared": lambda L, a, b, y, M, N: L.nvfp4_gemm_prepared(a, a, b, b, A, None, y, M, N, 24, S),
    "nvfp4_gemm_quantize_out": lambda L, a, b, y, M, N: L.nvfp4_gemm_quantize_out(
        a, a, b, b, A, None, A, y, y, M, N, 24, S),
    "nvfp4_debug_gemm_f32": lambda L, a, b, y, M, N: L.nvfp4_debug_gemm_f32(
        a, a, b, b, 0, A, None, y, M, N, 24, S),
    "int8_gemm": lambda L, a, b, y, M, N: L.int8_gemm(a, a, b, b, None, y, M, N, 24, S),
    "nvfp4_linear": lambda L, a, b, y, M, N: L.nvfp4_linear(
        a, M, 24, b, b, A, N, None, None, 0, A, 1 << 20, y, S),
    "nvfp4_linear_prepared": lambda L, a, b, y, M, N: L.nvfp4_linear_prepared(
        a, M, 24, b, b, A, N, None, None, 0, A, 1 << 20, y, S),
    "nvfp4_linear_fixed_scratch": lambda L, a, b, y, M, N: L.nvfp4_linear_fixed_scratch(
        a, M, 24, b, b, A, N, None, None, 0, y, S),
    "int8_linear": lambda L, a, b, y, M, N: L.int8_linear(a, M, 24, b, b, N, None, A, 1 << 20, y, S),
    "nvfp4_gemm_act": lambda L, a, b, y, M, N: L.nvfp4_gemm_act(
        a, a, b, b, 0, A, None, 2, None, y, M, N, 24, S),
    "int8_gemm_act": lambda L, a, b, y, M, N: L.int8_gemm_act(a, a, b, b, None, 2, None, y, M, N, 24, S),
    "nvfp4_linear_act": lambda L, a, b, y, M, N: L.nvfp4_linear_act(
        a, M, 24, b, b, 0, A, N, None, None, 0, 2, None, A, 1 << 20, y, S),
    "int8_linear_act": lambda L, a, b, y, M, N: L.int8_linear_act(
        a, M, 24, b, b, N, None, 2, None, A, 1 << 20, y, S),
}


@pytest.mark.parametrize("name", PRODUCTS)
def test_products_of_no_rows_or_columns(L, name):
    f = PRODUCTS[name]
    assert f(L, None, A, None, 0, 8) == SHAPE
    assert f(L, A, None, None, 8, 0) == SHAPE
    assert f(L, None, None, None, 0, 0) == SHAPE
    assert f(L, None, A, A, 8, 8) == INVALID
    assert f(L, A, None, A, 8, 8) == INVALID
    assert f(L, A, A, None, 8, 8) == INVALID
    assert f(L, None, A, None, 8, 0) == INVALID           # the activation has rows
    assert f(L, A, None, None, 0, 8) == INVALID           # the weight has columns
    assert f(L, None, None, None, -1, 8) == INVALID
