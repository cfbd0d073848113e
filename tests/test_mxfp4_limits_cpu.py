"""Bounds of the MXFP4 calls at the ends of 32 bits; they answer without a GPU and touch no pointer."""
import ctypes

import pytest

import group_gemm_gb300 as gg

P = ctypes.c_void_p(1 << 20)      # aligned, never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    gg.build()
    return gg.load()


@pytest.mark.parametrize("n", [2 ** 31 - 8, 2 ** 31 - 64, 2 ** 31 - 120])
def test_weight_quantiser_refuses_widths_whose_column_count_overflows(lib, n):
    """(n + 127) / 128 column atoms, counted in 32 bits by the kernel, leave them above 2^31 - 128."""
    assert lib.rdot_quantize_mxfp4_weight(P, gg.RDOT_BF16, 1, 32, n, P, P, None, None) == gg.RDOT_ERR_UNSUPPORTED
