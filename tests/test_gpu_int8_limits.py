"""The 8-bit integer product at its limits where the operands change places: as many tokens as a
launch holds, and more."""

import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from parity_util import DEV

pytestmark = pytest.mark.gpu


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
