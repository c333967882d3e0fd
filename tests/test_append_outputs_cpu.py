"""What an append writes shares no memory: the caches of keys and values and their scales stand apart, as
do the slots (no GPU: refused before any HIP call)."""

import pytest
import torch

from fp8_quantized_gemm_amax_amd import serving
from test_rope_abi_cpu import ROPE, four, rope
from test_serving_abi_cpu import A, APPEND, E4M3, SAME, SHAPE, b16, cache, call, ints

MXFP4 = serving.FP8_KV_MXFP4
# 4 pages of 2 heads, 16 tokens and 128 channels: 128 rows
CODES, SCALES = {SAME: 32768, E4M3: 16384, MXFP4: 8192}, {SAME: 0, E4M3: 512, MXFP4: 512}


@pytest.mark.parametrize("name,base", [("fp8_kv_append", APPEND), ("fp8_rope_append", ROPE)])
@pytest.mark.parametrize("fmt", [SAME, E4M3, MXFP4])
def test_entry_points_refuse_caches_that_share_memory(fmt, name, base):
    B = 1 << 24                                                        # places far from each other
    apart = dict(v=A + 4096, kc=B, vc=2 * B, ks=3 * B, vs=4 * B)
    if fmt == SAME:
        apart.update(ks=None, vs=None)
    for at, to in (("vc", B), ("vc", B + CODES[fmt] - 16), ("kc", 2 * B + CODES[fmt] - 16)):
        assert call(name, base, fmt=fmt, **dict(apart, **{at: to})) == SHAPE
    if fmt != SAME:
        for at, to in (("vs", 3 * B), ("vs", 3 * B + SCALES[fmt] - 4), ("ks", B), ("vs", 2 * B + CODES[fmt] - 4), ("ks", 2 * B + 64), ("vc", 3 * B + SCALES[fmt] - 16)):
            assert call(name, base, fmt=fmt, **dict(apart, **{at: to})) == SHAPE


def test_binding_refuses_caches_that_share_memory():
    k, slots = b16(3, 2, 64), ints(3).long()
    c, x = cache(), four(32)
    s = four(2)
    pair = torch.zeros(2 * c.numel() - 64, dtype=c.dtype)
    last = pair[-c.numel():].view(c.shape)
    for kc, vc, kw in ((c, c, {}), (pair[:c.numel()].view(c.shape), last, {}), (x, x, dict(k_scales=s, v_scales=four(2))), (x, four(32), dict(k_scales=s, v_scales=s)),
                       (x, four(32), dict(k_scales=x.view(-1)[:256].view(4, 2, 16, 2), v_scales=s))):
        with pytest.raises(ValueError, match="overlap"):
            rope(serving, kc=kc, vc=vc, **kw)
        with pytest.raises(ValueError, match="overlap"):
            serving.fp8_kv_append(k, k.clone(), slots, kc, vc, kw.get("k_scales"), kw.get("v_scales"))


def test_binding_refuses_slots_in_a_cache():
    c = cache()
    with pytest.raises(ValueError, match="overlap"):
        serving.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), c.view(-1).view(torch.int64)[:3], c, cache())
