"""The 8-bit integer product at its limits where the operands change places: K at its limit for up to 16
output channels, and as many tokens as a launch holds, and more."""

import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from parity_util import DEV
from test_gpu_int8 import check_gemm, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [17, 40, 200])
@pytest.mark.parametrize("N", [1, 2, 16])
def test_largest_sums_of_few_channels(N, M):
    """Codes of -128 and 127 only at K = 131056: sums up to 2^31 - 2^18, exact."""
    K = 131056
    assert fp8.fp8_debug_gemm_plan("int8", M, N, K)[0]["swapped"]
    qa, sa, qb, sb = operands(M, N, K, seed=M)
    qa[:], qb[:] = -128, -128
    qb[1::2] = 127
    qa[M // 2:, ::3] = 127
    assert int(qa[0].long() @ qb[0].long()) == 128 * 128 * K
    check_gemm((qa, sa, qb, sb), "bf16")


@pytest.mark.parametrize("M", [2 ** 26 - 4, 2 ** 26 + 5])
def test_one_channel_of_as_many_tokens_as_a_launch_holds_and_more(M):
    K = 16
    assert fp8.fp8_debug_gemm_plan("int8", M, 1, K)[0]["swapped"] == (M < 2 ** 26)
    g = torch.Generator(device=DEV).manual_seed(1)
    qa, qb = (torch.randint(-128, 128, (r, K), generator=g, dtype=torch.int8, device=DEV) for r in (M, 1))
    sa, sb = (torch.rand(r, generator=g, device=DEV) * 0.02 + 1e-3 for r in (M, 1))
    full = torch.full((M + 512, 1), -7.0, dtype=torch.bfloat16, device=DEV)
    fp8.int8_gemm_scaled_rowwise(qa, sa, qb, sb, out=full[:M])
    torch.cuda.synchronize()
    assert (full[M:] == -7.0).all()
    sums = torch.zeros(M, dtype=torch.int32, device=DEV)
    for k in range(K):
        sums += qa[:, k].int() * qb[0, k].int()
    assert torch.equal(full[:M, 0], (sums.float() * (sa * sb)).bfloat16())
