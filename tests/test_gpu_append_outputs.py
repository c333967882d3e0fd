"""An append into caches and scales that are neighbours in memory."""

import pytest
import torch

from fp8_quantized_gemm_amax_amd import serving

pytestmark = pytest.mark.gpu
SAME, E4M3, MXFP4 = serving.FP8_KV_SAME, serving.FP8_KV_E4M3, serving.FP8_KV_MXFP4


@pytest.mark.parametrize("fmt", [SAME, E4M3, MXFP4])
def test_neighbours_are_apart(fmt):
    """Caches and scales that lie one behind the other in one allocation, as a serving program may hold them."""
    tokens, hk, dim, page, pages = 20, 2, 64, 16, 3
    kind, width = (torch.bfloat16, dim) if fmt == SAME else (torch.uint8, dim if fmt == E4M3 else dim // 2)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.empty((tokens, hk, dim), device="cuda").normal_(generator=g).bfloat16() for _ in "kv")
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
    results = []
    for together in (False, True):
        codes = torch.zeros((2, pages, hk, page, width), dtype=kind, device="cuda")
        scales = torch.zeros((2, pages, hk, page) + (() if fmt == E4M3 else (dim // 32,)), dtype=torch.float32 if fmt == E4M3 else torch.uint8, device="cuda")
        parts = [*codes, *(scales if fmt != SAME else (None, None))]
        if not together:
            parts = [p if p is None else p.clone() for p in parts]
        serving.fp8_kv_append(k, v, slots, *parts)
        results.append([p for p in parts if p is not None])
    assert all(torch.equal(a, b) for a, b in zip(*results)) and all(p.any() for p in results[0])


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("fmt", [SAME, E4M3, MXFP4])
def test_one_cache_for_keys_and_values_that_are_one(fmt, strided):
    """The same tensor as k and v into the same cache, also where it has to be copied first."""
    tokens, hk, dim, page, pages = 20, 2, 64, 16, 3
    kind, width = (torch.bfloat16, dim) if fmt == SAME else (torch.uint8, dim if fmt == E4M3 else dim // 2)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((tokens, hk, dim + 4), device="cuda").normal_(generator=g).bfloat16()[..., :dim]
    if not strided:
        x = x.contiguous()
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]

    def parts():
        codes = torch.zeros((pages, hk, page, width), dtype=kind, device="cuda")
        scales = None if fmt == SAME else torch.zeros((pages, hk, page) + (() if fmt == E4M3 else (dim // 32,)), dtype=torch.float32 if fmt == E4M3 else torch.uint8, device="cuda")
        return codes, scales

    (k, ks), (v, vs), (c, s) = parts(), parts(), parts()
    serving.fp8_kv_append(x, x.clone(), slots, k, v, ks, vs)
    serving.fp8_kv_append(x, x, slots, c, c, s, s)
    assert torch.equal(c, k) and torch.equal(c, v) and (s is None or torch.equal(s, ks)) and c.any()
    with pytest.raises(ValueError, match="overlap"):
        serving.fp8_kv_append(x, x.clone(), slots, c, c, s, s)
    if s is not None:
        with pytest.raises(ValueError, match="overlap"):
            serving.fp8_kv_append(x, x, slots, c, c, s, vs)
