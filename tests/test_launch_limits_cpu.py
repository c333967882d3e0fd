"""Products whose launch would need 2^32 threads or more are refused as too large before anything else is
looked at (no GPU): with null pointers, one shape on either side of each limit."""

import pytest

import fp8_quantized_gemm_amax_amd as fp8
from fp8_quantized_gemm_amax_amd import int8
from fp8_quantized_gemm_amax_amd.binding import lib

# rows, channels at the limit, K: one token takes 64 threads a channel, 5 to 16 tokens 256 for 32 channels, 17 to 128
# 512 for 112, more than that 512 for a tile of 256 x 256
SHAPES = [(1, 2 ** 26 - 4, 128), (7, 2 ** 29 - 32, 128), (100, 112 * (2 ** 23 - 1), 128), (2 ** 31 - 256, 256, 128)]


def product(mode, *shape):
    if mode == "int8":
        code = int8._lib()["int8_gemm_scaled_rowwise"](None, None, None, None, *shape, None, 0, None)
    else:
        code = getattr(lib(), "fp8_gemm_scaled_" + mode)(None, None, None, None, *shape, None, 0, None)
    return fp8.binding.STATUS_NAMES[code]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("mode", ["tensorwise", "blockwise", "blockwise_ue8m0", "rowwise", "int8"])
def test_products(mode, M, N, K):
    assert product(mode, M, N, K) == "FP8_ERR_NULL_POINTER"
    more = (M + 1, N) if M > N else (M, N + 1)
    assert product(mode, *more, K) == "FP8_ERR_TOO_LARGE"


@pytest.mark.parametrize("mode", range(4))
def test_one_token_step(mode):
    def step(N, K):
        return fp8.binding.STATUS_NAMES[lib().fp8_gemv_dynamic(mode, None, 0, None, None, N, K, None, None, None, 0, None)]
    assert step(2 ** 26 - 4, 128) == "FP8_ERR_NULL_POINTER"
    assert step(2 ** 26 - 3, 128) == "FP8_ERR_TOO_LARGE"
    if mode in (0, 3):                                   # in one launch, whose waves take many channels
        assert step(2 ** 27 - 1, 16) == "FP8_ERR_NULL_POINTER"
