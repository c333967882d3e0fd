"""Rotation with append and the four-bit caches, host side (no GPU): the C entry points and the Python
binding refuse bad arguments before any HIP call."""

import pytest
import torch

from fp8_quantized_gemm_amax_amd import serving
from test_serving_abi_cpu import A, APPEND, PAGED, SHAPE, ALIGN, DTYPE, LARGE, NULLP, OK, b16, cache, call, ints

T, V = TypeError, ValueError
MXFP4 = serving.FP8_KV_MXFP4
ROPE = dict(q=A, k=A, v=A, dt=0, tokens=4, hq=8, hk=2, dim=128, qts=1024, qhs=128, kts=256, khs=128, vts=256, vhs=128, positions=A, turn=A,
            n_positions=100, rotary=128, interleaved=0, slots=A, pages=4, page=16, fmt=MXFP4, kc=A, vc=A, ks=A, vs=A, out=A, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), SHAPE), (dict(hq=-1), SHAPE), (dict(hk=0), SHAPE), (dict(dim=96), SHAPE), (dict(page=17), SHAPE), (dict(pages=0), SHAPE),
    (dict(rotary=0), SHAPE), (dict(rotary=-16), SHAPE), (dict(rotary=24), SHAPE), (dict(rotary=144), SHAPE), (dict(rotary=8), SHAPE),
    (dict(n_positions=-1), SHAPE), (dict(dt=2), DTYPE), (dict(fmt=2), DTYPE), (dict(fmt=-1), DTYPE), (dict(kts=-8), SHAPE), (dict(qts=-8), SHAPE),
    (dict(qhs=4), ALIGN), (dict(vhs=129), ALIGN), (dict(tokens=2 ** 31), LARGE), (dict(hk=65536), LARGE), (dict(hq=65536), LARGE),
    (dict(n_positions=2 ** 31), LARGE), (dict(tokens=2 ** 26, hq=32), LARGE), (dict(qts=2 ** 40), LARGE), (dict(pages=2 ** 36), LARGE),
    (dict(q=None), NULLP), (dict(out=None), NULLP), (dict(k=None), NULLP), (dict(positions=None), NULLP), (dict(turn=None), NULLP),
    (dict(slots=None), NULLP), (dict(vs=None), NULLP), (dict(kc=None), NULLP), (dict(q=A + 8), ALIGN), (dict(out=A + 2), ALIGN),
    (dict(positions=A + 2), ALIGN), (dict(turn=A + 4), ALIGN), (dict(ks=A + 1), ALIGN), (dict(slots=A + 4), ALIGN), (dict(vc=A + 8), ALIGN),
    (dict(tokens=0), OK), (dict(tokens=0, q=None, k=None), OK)])
def test_rope_refusals(change, status):
    assert call("fp8_rope_append", ROPE, **change) == status


def test_rope_without_queries_asks_nothing_of_them():
    assert call("fp8_rope_append", ROPE, hq=0, q=None, out=None, qts=3, qhs=-7, positions=None) == NULLP      # the next check


@pytest.mark.parametrize("dim,heads,each", [(128, 1, 16), (64, 1, 32)])
def test_more_work_than_a_launch_holds_is_too_large(dim, heads, each):
    """A workgroup takes 32 (64) units of a token; without queries a key head is one, so fp8_kv_append's limit holds first."""
    limit = (2 ** 24 - 1) * each
    base = dict(hk=heads, hq=0, dim=dim, rotary=64, kts=dim, vts=dim, khs=0, vhs=0, k=None)
    assert call("fp8_rope_append", ROPE, **base, tokens=limit) == NULLP
    assert call("fp8_rope_append", ROPE, **base, tokens=limit + 1) == LARGE


@pytest.mark.parametrize("name,base", [("fp8_kv_append", APPEND), ("fp8_attn_paged", PAGED)])
def test_four_bits_take_any_scale_bytes_from_four_byte_addresses(name, base):
    assert call(name, base, fmt=MXFP4, ks=None) == NULLP
    assert call(name, base, fmt=MXFP4, vs=A + 2) == ALIGN
    assert call(name, base, fmt=MXFP4, kc=None) == NULLP


def rope(s, q=b16(3, 4, 64), k=b16(3, 2, 64), v=b16(3, 2, 64), positions=ints(3), turn=torch.zeros(9, 64), slots=ints(3).long(), kc=None, vc=None, **kw):
    return s.fp8_rope_append(q, k, v, positions, turn, slots, cache() if kc is None else kc, cache() if vc is None else vc, **kw)


U8 = torch.uint8


def four(*tail):
    return torch.zeros((4, 2, 16, *tail), dtype=U8)


@pytest.mark.parametrize("error,match,change", [
    (V, "like k", dict(v=b16(3, 2, 64).half())),
    (T, "k must be bfloat16", dict(k=b16(3, 2, 64).float())),
    (T, "q must be of k's type", dict(q=b16(3, 4, 64).half())),
    (V, "q has 2 tokens", dict(q=b16(2, 4, 64))),
    (V, "q must have head_dim 64", dict(q=b16(3, 4, 128))),
    (V, "k has 1 heads", dict(k=b16(3, 1, 64), v=b16(3, 1, 64))),
    (T, "positions must be Int", dict(positions=ints(3).long())),
    (V, "positions must have shape", dict(positions=ints(2))),
    (T, "cos_sin must be Float", dict(turn=torch.zeros(9, 64).double())),
    (V, "cos_sin must be .positions", dict(turn=torch.zeros(9))),
    (V, "cos_sin must be contiguous", dict(turn=torch.zeros(64, 9).t())),
    (V, "rotary_dim", dict(turn=torch.zeros(9, 24))),
    (V, "rotary_dim", dict(turn=torch.zeros(9, 80))),
    (T, "slots must be Long", dict(slots=ints(3))),
    (V, "out goes with q", dict(q=None, out=b16(3, 4, 64))),
    (V, "out must have shape", dict(out=b16(3, 4, 32))),
    (T, "out must be", dict(out=b16(3, 4, 64).half())),
    (T, "k must be a tensor", dict(k=None)),
    (RuntimeError, "ambiguous", dict(interleaved=torch.zeros(2))),
    (V, "k_scales must have shape", dict(kc=four(32), vc=four(32), k_scales=four(1), v_scales=four(1))),
    (V, "v_scales must have shape", dict(kc=four(32), vc=four(32), k_scales=four(2), v_scales=four(1))),
    (V, "go together", dict(kc=four(32), vc=four(32), k_scales=four(2))),
    (V, "head_dim 128", dict(kc=four(64), vc=four(64), k_scales=four(4), v_scales=four(4))),
    (T, "v_scales must be", dict(kc=four(32), vc=four(32), k_scales=four(2), v_scales=four(2).float())),
    (T, "scales of a byte", dict(k_scales=four(2), v_scales=four(2))),
    (V, "on the GPU", dict()),
    (V, "on the GPU", dict(q=None)),
    (V, "on the GPU", dict(kc=four(32), vc=four(32), k_scales=four(2), v_scales=four(2))),
])
def test_binding_refuses(error, match, change):
    with pytest.raises(error, match=match):
        rope(serving, **change)


def test_binding_refuses_tensors_that_share_memory():
    x = b16(3, 8, 64)
    with pytest.raises(ValueError, match="out overlaps"):
        rope(serving, q=x[:, :4], out=x.view(-1)[:768].view(3, 4, 64))
    c = cache()
    with pytest.raises(ValueError, match="cache overlaps"):
        rope(serving, k=c.view(-1)[:384].view(3, 2, 64), kc=c)
    with pytest.raises(ValueError, match="out overlaps"):
        rope(serving, kc=c, out=c.view(-1)[:768].view(3, 4, 64))


def test_rope_table():
    t = serving.rope_table(5, 32, base=100.0, device="cpu")
    assert t.shape == (5, 32) and t.dtype == torch.float32
    want = torch.arange(5).double()[:, None] * 100.0 ** (-torch.arange(16).double() / 16)
    assert torch.equal(t, torch.cat([want.cos(), want.sin()], 1).float())
    for bad in ((5, 0), (5, 31), (-1, 32)):
        with pytest.raises(ValueError):
            serving.rope_table(*bad, device="cpu")
