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


@pytest.mark.parametrize("batch,q_len,heads", [(2 ** 30, 2 ** 24, 2 ** 10), (2 ** 30, 2 ** 20, 2 ** 14), (2 ** 24, 2 ** 24, 2 ** 17),
                                               (2 ** 31 - 1, 2 ** 24, 2 ** 30)])
def test_query_rows_whose_number_leaves_64_bits(lib, batch, q_len, heads):
    """Their product wraps to zero or below."""
    s = (ctypes.c_longlong * 3)(2 ** 35, 64, 64)
    a = kb.ScoredAttention(P, P, P, 2 * P, None, None, None, None, None, None, s, s, s, s, batch, q_len, 8, heads, heads,
                           64, kb.BF16, 0, 0.125, 0.0)
    n = ctypes.c_size_t(77)
    for rc in (lib.kimodo_attention_scored(ctypes.byref(a), None, 0, None),
               lib.kimodo_attention_scored_workspace(ctypes.byref(a), ctypes.byref(n))):
        assert rc == -1, rc
        assert b"too many query rows" in lib.kimodo_last_error()
