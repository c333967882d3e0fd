"""Attention over a paged cache where requests and rows must not reach each other: pages that do not
exist next to scales that are not finite, value scales far apart, and keys and values that are not
finite in places that some rows see and others do not.  Float64 references as in test_gpu_serving.py."""

import math

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from oracle import decode_e4m3
from oracle.serving import attention_ref
from parity_util import DEV
from serving_util import Cache, check_rows, cu_of, f64_of, normal

pytestmark = pytest.mark.gpu


def set_row(cache, name, r, token, codes=None, scale=None):
    """Overwrites a token of request r in an e4m3 cache (every head): its codes, its scale."""
    page, at = int(cache.table[r, token // cache.page]), token % cache.page
    if codes is not None:
        getattr(cache, name)[page, :, at] = codes
    if scale is not None:
        getattr(cache, name + "s")[page, :, at] = scale


def reread(cache):
    """The cache's values from what its tensors hold now."""
    for n in "kv":
        c, s = (x.cpu().numpy() for x in (getattr(cache, n), getattr(cache, n + "s")))
        cache.values[n] = decode_e4m3(c).astype(np.float64) * s.astype(np.float64)[..., None]


# ------------------------------------------------- several requests of one workgroup, e4m3 scales

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_missing_pages_next_to_scales_that_are_not_finite(dim, dtype):
    """More requests than workgroups, so that a workgroup takes several: every second request has a key and
    a value whose scale is NaN or infinite, the others lack the page at the same place, which reads as zero."""
    batch, n, page, hk = 700, 70, 16, 2
    cache = Cache([n] * batch, hk, dim, page, dtype, True, 3, width=20)
    table = cache.dev_table.clone()
    odd = list(range(1, batch, 2))
    for r in range(0, batch, 2):
        bad = (float("nan"), float("inf"))[r // 2 % 2]
        for token in (20, 66):
            set_row(cache, "kv"[r // 4 % 2], r, token, scale=bad)
    table[odd, 1] = -1
    table[odd, 4] = 1 << 30
    q = normal((batch, 4 * hk, dim), dtype, 4)
    out = fp8.fp8_attn_paged(q, cache.k, cache.v, table, cache.dev_lens, cu_of([1] * batch), cache.ks, cache.vs, max_new=1)
    assert out[odd].isfinite().all()
    for r in odd[:60:7] + odd[-40::7]:
        kk, vv = cache.request("k", r).copy(), cache.request("v", r).copy()
        for x in (kk, vv):
            x[16:32], x[64:70] = 0, 0
        ref = attention_ref(f64_of(q[r:r + 1]), kk, vv, n - 1, 1 / math.sqrt(dim), 0)
        check_rows(out[r:r + 1], None, ref, dtype, n, dim, float(np.abs(vv).max()), f"request {r}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_requests_whose_value_scales_lie_far_apart(dim, dtype):
    """Neighbours in a workgroup with value scales 2^14 apart: each is as exact as it is alone, bit for bit."""
    batch, page, hk = 700, 16, 2
    lens = [180 if r % 2 else 200 for r in range(batch)]
    cache = Cache(lens, hk, dim, page, dtype, True, 5, width=20)
    for r in range(0, batch, 2):
        pages = torch.from_numpy(cache.table[r, : -(-lens[r] // page)].astype(np.int64)).to(DEV)
        cache.vs[pages] *= 2.0 ** 14
    reread(cache)
    q = normal((batch, 4 * hk, dim), dtype, 6)
    args = (cache.k, cache.v)
    out = fp8.fp8_attn_paged(q, *args, cache.dev_table, cache.dev_lens, cu_of([1] * batch), cache.ks, cache.vs, max_new=1)
    for r in (1, 2, 3, 301, 303, 699):
        kk, vv = cache.request("k", r), cache.request("v", r)
        ref = attention_ref(f64_of(q[r:r + 1]), kk, vv, lens[r] - 1, 1 / math.sqrt(dim), 0)
        check_rows(out[r:r + 1], None, ref, dtype, lens[r], dim, 0.0, f"request {r}")
        alone = fp8.fp8_attn_paged(q[r:r + 1], *args, cache.dev_table[r:r + 1, :13].contiguous(), cache.dev_lens[r:r + 1], cu_of([1]),
                                   cache.ks, cache.vs, max_new=1)
        assert torch.equal(out[r:r + 1], alone), r
