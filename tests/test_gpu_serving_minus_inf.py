"""A key whose score is -infinity for some rows and a value of the same token that is not finite: a row that
sees the token gets what the value holds under any weight, 0 too, and other channels and the rows before the
token keep their bits."""

import math

import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from mxfp4_util import Cache4
from parity_util import DEV
from serving_util import Cache, cu_of, normal

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def spoil(cache, fmt, page, at):
    """Token (page, at) of key head 1: a key of zeros but for channel 0, which is +infinity, and values that are not finite
    in the channels that are returned."""
    if fmt == "mxfp4":
        cache.k[page, 1, at] = 0
        cache.k[page, 1, at, 0], cache.ks[page, 1, at, 0] = 2, 160        # 2^33: infinite in fp16
        cache.vs[page, 1, at, 1] = 255
        return slice(32, 64)
    cache.k[page, 1, at] = 0
    if fmt == "e4m3":
        cache.k[page, 1, at, 0], cache.ks[page, 1, at] = 0x38, math.inf   # 1 times infinity
        cache.vs[page, 1, at] = math.nan
        return slice(0, None)
    cache.k[page, 1, at, 0] = math.inf
    cache.v[page, 1, at, 5] = -math.inf
    return slice(5, 6)


@pytest.mark.parametrize("fmt,dtype", [("same", "bf16"), ("same", "f16"), ("e4m3", "bf16"), ("e4m3", "f16"), ("mxfp4", "f16")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [3, 14, 90])
@pytest.mark.parametrize("length", [130, 3000])
def test_paged(length, new, dim, fmt, dtype):
    q = normal((new, 8, dim), dtype, 31)
    q[:, :, 0] = torch.where(torch.arange(new * 8, device=DEV).view(new, 8) % 3 > 0, -1.0, 1.0)      # scores of -inf and +inf
    cache = Cache4([length], 2, dim, 16, 32) if fmt == "mxfp4" else Cache([length], 2, dim, 16, dtype, fmt == "e4m3", 32)

    def run():
        return fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of([new]), cache.ks, cache.vs, max_new=new)

    if fmt == "same":
        cache.ks = cache.vs = None
    good = run()
    token = length - 2
    channels = spoil(cache, fmt, int(cache.table[0, token // 16]), token % 16)
    out = run()
    assert same(out[:-2], good[:-2]) and same(out[:, :4], good[:, :4])     # rows before it, and the other key head
    assert not out[-2:, 4:, channels].isfinite().any()
    below = q[-2:, 4:, 0] < 0                                              # no weight in the other channels
    keep = [c for c in range(dim) if c not in range(dim)[channels]]
    assert out[-2:, 4:][below][:, keep].isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length", [40, 700])
def test_prompt(length, dim, dtype):
    q, k, v = (normal((length, h, dim), dtype, 33 + i) for i, h in enumerate((4, 2, 2)))
    q[:, :, 0] = torch.where(torch.arange(length * 4, device=DEV).view(length, 4) % 3 > 0, -1.0, 1.0)
    good = fp8.fp8_attn_prompt(q, k, v, cu_of([length]))
    at = length // 2
    k[at, 1] = 0.0
    k[at, 1, 0], v[at, 1, 7] = math.inf, math.nan
    out = fp8.fp8_attn_prompt(q, k, v, cu_of([length]))
    assert same(out[:at], good[:at]) and same(out[:, :2], good[:, :2])
    assert out[at:, 2:, 7].isnan().all()
    assert out[at:, 2:][q[at:, 2:, 0] < 0][:, :7].isfinite().all()
