"""The workspace that attention over a paged cache asks for, host side (no GPU): a size that the query
tells serves every format, and a format is not refused for what another one needs."""

import pytest

from fp8_quantized_gemm_amax_amd import serving
from test_serving_abi_cpu import E4M3, NULLP, PAGED, SAME, SHAPE, call, fns

MXFP4 = serving.FP8_KV_MXFP4


@pytest.mark.parametrize("heads", [8, 512, 513, 1024])
def test_many_key_heads(heads):
    """Up to 1024 partial results of 32 rows; four bits leave two a key head, more than that from 513 heads on."""
    def need(heads):
        return fns()["fp8_attn_paged_workspace"](4, 4, heads, heads, 64, 64, 16, 1)

    def refused(fmt, ws_bytes):
        status = call("fp8_attn_paged", PAGED, tokens=4, batch=4, hq=heads, hk=heads, dim=64, width=64, max_new=1, fmt=fmt, ws_bytes=ws_bytes, ws=None)
        assert status in (SHAPE, NULLP)
        return status == SHAPE

    assert need(512) == need(8) == 16384 + 16 + 16 * 4096 + 4096 * 32 * 8 + 1024 * 32 * 64 * 4
    for fmt in (SAME, E4M3, MXFP4):
        assert not refused(fmt, need(heads)) and refused(fmt, need(8) - 1)
    assert not refused(SAME, need(8)) and not refused(E4M3, need(8))
    assert refused(MXFP4, need(8)) == (heads > 512) and refused(MXFP4, need(heads) - 1)
