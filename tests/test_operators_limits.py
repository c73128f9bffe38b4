"""Sizes near the ends of 32 and 64 bits are refused on the host: the kernels count rows and tiles in
32-bit integers, which would wrap there and pass their own checks."""
import ctypes

import pytest

import transformer_denoiser_b200 as kb

P = 4096   # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    from transformer_denoiser_b200.build import build
    build()
    return kb.load_library()


@pytest.mark.parametrize("M,N", [(2 ** 31 - 1, 1), (2 ** 31 - 512, 8), (1, 2 ** 31 - 1), (8, 2 ** 31 - 512)])
@pytest.mark.parametrize("epi", [0, 1, 2, 3])
def test_products_of_nearly_2_31_rows(lib, M, N, epi):
    """The last tile's end lies past 2^31: a row index that wraps below zero is below M."""
    rc = lib.kimodo_gemm_int8(P, 16, P, 2 * P, 16, P, None, P, N, 3 * P, N, M, N, 16, epi, 1 if epi == 3 else 0, None)
    assert rc == -1, rc
    assert b"at most 2147483135" in lib.kimodo_last_error()
