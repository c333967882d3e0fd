"""The serving operators' host side (no GPU): every entry point include/fp8amax_serving.h
declares is exported and bound, refuses bad arguments with the documented status before any
HIP call, and the Python binding refuses tensors of the wrong type, shape, order or device."""

import ctypes
import os
import re

import pytest
import torch

from fp8_quantized_gemm_amax_amd import serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLP, SHAPE, DTYPE, ALIGN, LAUNCH, LARGE = range(7)
A = 0x10000            # fake, aligned addresses (never dereferenced: validation fails first)
BF16, SAME, E4M3 = 0, 0, 1


def fns():
    return serving._lib()


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "fp8amax_serving.h")).read()
    names = re.findall(r"^(?:fp8_status_t|int64_t)\s+(fp8_\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(serving._SIGNATURES) == set(fns())


PLAN = dict(cached=A, added=A, batch=4, page=16, table=A, width=8, free=A, n_free=5, taken=A, tokens=10, cu=A, lens=A,
            positions=A, slots=A, taken_out=A + 64, missing=A, stream=None)
APPEND = dict(k=A, v=A, dt=BF16, tokens=4, heads=2, dim=128, kts=256, khs=128, vts=256, vhs=128, slots=A, pages=4,
              page=16, fmt=E4M3, kc=A, vc=A, ks=A, vs=A, stream=None)
PROMPT = dict(q=A, k=A, v=A, dt=BF16, tokens=4, cu=A, batch=2, hq=8, hk=2, dim=128, qts=1024, qhs=128, kts=256, khs=128,
              vts=256, vhs=128, scale=0.1, window=0, out=A, lse=None, stream=None)
PAGED = dict(q=A, dt=BF16, tokens=4, cu=A, batch=2, hq=8, hk=2, dim=128, qts=1024, qhs=128, fmt=E4M3, kc=A, vc=A, ks=A,
             vs=A, pages=8, page=16, table=A, width=4, lens=A, scale=0.1, window=0, max_new=0, out=A, lse=None, ws=A,
             ws_bytes=1 << 40, stream=None)


def call(name, base, **change):
    return fns()[name](*dict(base, **change).values())


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(n_free=-1), SHAPE), (dict(width=0), SHAPE),
    (dict(page=8), SHAPE), (dict(page=24), SHAPE), (dict(page=2048), SHAPE), (dict(page=0), SHAPE), (dict(page=-16), SHAPE),
    (dict(batch=16385), LARGE), (dict(tokens=2 ** 31), LARGE), (dict(width=2 ** 28), LARGE), (dict(n_free=2 ** 31), LARGE),
    (dict(cached=None), NULLP), (dict(table=None), NULLP), (dict(free=None), NULLP), (dict(taken=None), NULLP),
    (dict(cu=None), NULLP), (dict(slots=None), NULLP), (dict(missing=None), NULLP), (dict(lens=None), NULLP),
    (dict(added=A + 2), ALIGN), (dict(slots=A + 4), ALIGN), (dict(taken_out=A), SHAPE),
])
def test_plan_refusals(change, status):
    assert call("fp8_paged_plan", PLAN, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), SHAPE), (dict(heads=0), SHAPE), (dict(dim=96), SHAPE), (dict(dim=256), SHAPE), (dict(page=17), SHAPE),
    (dict(pages=0), SHAPE), (dict(dt=2), DTYPE), (dict(fmt=2), DTYPE), (dict(kts=-8), SHAPE), (dict(kts=4), ALIGN),
    (dict(vhs=129), ALIGN), (dict(tokens=2 ** 31), LARGE), (dict(heads=65536), LARGE), (dict(pages=2 ** 36), LARGE),
    (dict(kts=2 ** 40), LARGE), (dict(k=None), NULLP), (dict(slots=None), NULLP), (dict(ks=None), NULLP),
    (dict(vc=None), NULLP), (dict(k=A + 8), ALIGN), (dict(vc=A + 1), ALIGN), (dict(ks=A + 2), ALIGN), (dict(slots=A + 4), ALIGN),
    (dict(tokens=0), OK),
])
def test_append_refusals(change, status):
    assert call("fp8_kv_append", APPEND, **change) == status


ATTN = [
    (dict(tokens=-1), SHAPE), (dict(batch=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hk=0), SHAPE), (dict(hk=3), SHAPE),
    (dict(dim=80), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(window=-1), SHAPE), (dict(dt=3), DTYPE), (dict(qts=-8), SHAPE), (dict(qhs=3), ALIGN),
    (dict(tokens=2 ** 31), LARGE), (dict(hq=131072), LARGE), (dict(tokens=2 ** 28), LARGE), (dict(q=None), NULLP), (dict(cu=None), NULLP),
    (dict(out=None), NULLP), (dict(q=A + 2), ALIGN), (dict(out=A + 8), ALIGN), (dict(cu=A + 1), ALIGN), (dict(lse=A + 2), ALIGN),
    (dict(tokens=0), OK), (dict(batch=0), OK),
]


@pytest.mark.parametrize("change,status", ATTN + [
    (dict(kts=-8), SHAPE), (dict(vhs=4), ALIGN), (dict(kts=2 ** 21), LARGE), (dict(k=None), NULLP), (dict(v=A + 4), ALIGN)])
def test_prompt_refusals(change, status):
    assert call("fp8_attn_prompt", PROMPT, **change) == status


@pytest.mark.parametrize("change,status", ATTN + [
    (dict(fmt=7), DTYPE), (dict(page=20), SHAPE), (dict(pages=0), SHAPE), (dict(width=0), SHAPE), (dict(max_new=-1), SHAPE),
    (dict(width=2 ** 28), LARGE), (dict(kc=None), NULLP), (dict(vs=None), NULLP), (dict(table=None), NULLP),
    (dict(lens=None), NULLP), (dict(kc=A + 8), ALIGN), (dict(ks=A + 1), ALIGN), (dict(lens=A + 2), ALIGN)])
def test_paged_refusals(change, status):
    assert call("fp8_attn_paged", PAGED, **change) == status


def test_prompt_tokens_may_not_overlap():
    assert call("fp8_attn_prompt", PROMPT, kts=120) == SHAPE
    assert call("fp8_attn_prompt", PROMPT, vts=0) == SHAPE


def test_workspace_sizes():
    w = fns()["fp8_attn_paged_workspace"]
    assert w(4, 2, 8, 2, 128, 4, 16, 0) >= 0
    for bad in [(-1, 2, 8, 2, 128, 4, 16, 0), (4, 2, 8, 3, 128, 4, 16, 0), (4, 2, 8, 2, 96, 4, 16, 0), (4, 2, 8, 2, 128, 0, 16, 0),
                (4, 2, 8, 2, 128, 4, 10, 0), (4, 2, 8, 2, 128, 4, 16, -1)]:
        assert w(*bad) == 0
    need = w(64, 64, 32, 8, 128, 2048, 16, 1)
    assert need > 0
    if need:
        assert call("fp8_attn_paged", PAGED, tokens=64, batch=64, hq=32, hk=8, width=2048, max_new=1, ws_bytes=need - 1) == SHAPE
        assert call("fp8_attn_paged", PAGED, tokens=64, batch=64, hq=32, hk=8, width=2048, max_new=1, ws=None) == NULLP
        assert call("fp8_attn_paged", PAGED, tokens=64, batch=64, hq=32, hk=8, width=2048, max_new=1, ws=A + 4) == ALIGN


# ------------------------------------------------------------------------- the Python binding

def b16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def cache(dtype=torch.bfloat16):
    return torch.zeros((4, 2, 16, 64), dtype=dtype)


T, V = TypeError, ValueError


# The device is checked last, so every other refusal can be seen with tensors on the CPU.
@pytest.mark.parametrize("error,match,call", [
    (V, "added must have shape", lambda s: s.fp8_paged_plan(ints(3), ints(2), ints(3, 4), ints(5), ints(1), 3, 16)),
    (T, "cached must be Int", lambda s: s.fp8_paged_plan(ints(3).long(), ints(3), ints(3, 4), ints(5), ints(1), 3, 16)),
    (V, "block_table", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(2, 4), ints(5), ints(1), 3, 16)),
    (V, "block_table", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(4, 3).t(), ints(5), ints(1), 3, 16)),
    (T, "block_table", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(3, 4).long(), ints(5), ints(1), 3, 16)),
    (V, "taken must have shape", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(3, 4), ints(5), ints(2), 3, 16)),
    (V, "negative", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(3, 4), ints(5), ints(1), -1, 16)),
    (V, "page_size", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(3, 4), ints(5), ints(1), 3, 2 ** 40)),
    (T, "tokens must be an integer", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(3, 4), ints(5), ints(1), 3.5, 16)),
    (T, "cached must be a tensor", lambda s: s.fp8_paged_plan([1, 2, 3], ints(3), ints(3, 4), ints(5), ints(1), 3, 16)),
    (V, "out.positions must have shape", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(3, 4), ints(5), ints(1), 3, 16, out=s.paged_plan_buffers(3, 4, "cpu"))),
    (T, "PagedPlan", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(3, 4), ints(5), ints(1), 3, 16, out=ints(3))),
    (V, "like k", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64).half(), ints(3).long(), cache(), cache())),
    (T, "slots must be Long", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3), cache(), cache())),
    (V, "slots must have shape", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(4).long(), cache(), cache())),
    (V, "k has 1 heads", lambda s: s.fp8_kv_append(b16(3, 1, 64), b16(3, 1, 64), ints(3).long(), cache(), cache())),
    (V, "head_dim 64", lambda s: s.fp8_kv_append(b16(3, 2, 128), b16(3, 2, 128), ints(3).long(), cache(), cache())),
    (T, "without scales", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3).long(), cache(torch.float16), cache(torch.float16))),
    (T, "without scales", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3).long(), cache(torch.uint8), cache(torch.uint8))),
    (V, "go together", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3).long(), cache(torch.uint8), cache(torch.uint8), torch.ones(4, 2, 16))),
    (V, "k_scales must have shape", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3).long(), cache(torch.uint8), cache(torch.uint8), torch.ones(4, 2, 8), torch.ones(4, 2, 8))),
    (T, "k_scales must be Float", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3).long(), cache(torch.uint8), cache(torch.uint8), torch.ones(4, 2, 16).half(), torch.ones(4, 2, 16))),
    (T, "with scales", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3).long(), cache(), cache(), torch.ones(4, 2, 16), torch.ones(4, 2, 16))),
    (V, "k_cache must be contiguous", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3).long(), cache().transpose(1, 2).contiguous().transpose(1, 2), cache())),
    (T, "v_cache must be", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3).long(), cache(), cache(torch.float16))),
    (T, "q must be bfloat16", lambda s: s.fp8_attn_prompt(b16(3, 4, 64).float(), b16(3, 2, 64), b16(3, 2, 64), ints(2))),
    (V, "of q's type", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(3, 2, 64).half(), b16(3, 2, 64).half(), ints(2))),
    (V, "q has 3 tokens", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(4, 2, 64), b16(4, 2, 64), ints(2))),
    (V, "head_dim 64", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(3, 2, 128), b16(3, 2, 128), ints(2))),
    (V, "q must be .tokens", lambda s: s.fp8_attn_prompt(b16(3, 256), b16(3, 2, 64), b16(3, 2, 64), ints(2))),
    (T, "cu_tokens must be Int", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(3, 2, 64), b16(3, 2, 64), ints(2).long())),
    (V, "batch . 1 entries", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(3, 2, 64), b16(3, 2, 64), ints(0))),
    (T, "softmax_scale", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(3, 2, 64), b16(3, 2, 64), ints(2), softmax_scale="1")),
    (T, "window must be an integer", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(3, 2, 64), b16(3, 2, 64), ints(2), window=1.5)),
    (V, "out must have shape", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(3, 2, 64), b16(3, 2, 64), ints(2), out=b16(3, 4, 32))),
    (T, "out must be", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(3, 2, 64), b16(3, 2, 64), ints(2), out=b16(3, 4, 64).half())),
    (T, "v_cache must be", lambda s: s.fp8_attn_paged(b16(3, 4, 64), cache(), cache(torch.float16), ints(2, 4), ints(2), ints(3))),
    (V, "block_table", lambda s: s.fp8_attn_paged(b16(3, 4, 64), cache(), cache(), ints(3, 4), ints(2), ints(3))),
    (V, "cu_tokens must have shape", lambda s: s.fp8_attn_paged(b16(3, 4, 64), cache(), cache(), ints(2, 4), ints(2), ints(4))),
    (V, "head_dim 64", lambda s: s.fp8_attn_paged(b16(3, 4, 128), cache(), cache(), ints(2, 4), ints(2), ints(3))),
    (T, "without scales", lambda s: s.fp8_attn_paged(b16(3, 4, 64).half(), cache(), cache(), ints(2, 4), ints(2), ints(3))),
    (T, "without scales", lambda s: s.fp8_attn_paged(b16(3, 4, 64), cache(torch.uint8), cache(torch.uint8), ints(2, 4), ints(2), ints(3))),
    (V, "on the GPU", lambda s: s.fp8_paged_plan(ints(3), ints(3), ints(3, 4), ints(5), ints(1), 3, 16)),
    (V, "on the GPU", lambda s: s.fp8_kv_append(b16(3, 2, 64), b16(3, 2, 64), ints(3).long(), cache(), cache())),
    (V, "on the GPU", lambda s: s.fp8_attn_prompt(b16(3, 4, 64), b16(3, 2, 64), b16(3, 2, 64), ints(2))),
    (V, "on the GPU", lambda s: s.fp8_attn_paged(b16(3, 4, 64), cache(), cache(), ints(2, 4), ints(2), ints(3))),
])
def test_binding_refuses(error, match, call):
    with pytest.raises(error, match=match):
        call(serving)


def test_binding_refuses_tensors_that_share_memory():
    x = b16(3, 8, 64)
    with pytest.raises(ValueError, match="overlaps"):
        serving.fp8_attn_prompt(x[:, :4], x[:, 4:6], x[:, 6:], ints(2), out=x.view(-1)[:768].view(3, 4, 64))
    c = cache()
    k = c.view(-1)[:384].view(3, 2, 64)
    with pytest.raises(ValueError, match="overlaps"):
        serving.fp8_kv_append(k, b16(3, 2, 64), ints(3).long(), c, cache())
    plan = serving.paged_plan_buffers(3, 4, "cpu")
    with pytest.raises(ValueError, match="overlaps"):
        serving.fp8_paged_plan(plan.seq_lens, ints(3), ints(3, 4), ints(5), ints(1), 4, 16, out=plan)
    with pytest.raises(ValueError, match="overlaps"):
        serving.fp8_paged_plan(ints(3), ints(3), ints(3, 4), ints(5), ints(1), 3, 16, out=plan._replace(positions=plan.seq_lens, slots=ints(3).long()))


def test_enumerations_take_any_integer():
    """Unknown enumeration values are refused, not undefined."""
    assert call("fp8_kv_append", APPEND, dt=2 ** 31 - 1) == DTYPE
    assert call("fp8_attn_paged", PAGED, fmt=-1) == DTYPE
    assert ctypes.sizeof(ctypes.c_int) == 4


@pytest.mark.parametrize("name,base,most,change", [
    ("fp8_kv_append", APPEND, "tokens", dict(heads=1, dim=128)),                # 16 rows a workgroup
    ("fp8_kv_append", APPEND, "tokens", dict(heads=1, dim=64, kts=64, vts=64)),     # 32
    ("fp8_attn_prompt", PROMPT, "batch", dict(hq=1, hk=1)),                     # one a request, and one for 128 rows
    ("fp8_attn_paged", PAGED, "batch", dict(hq=1, hk=1)),
    ("fp8_attn_paged", PAGED, "batch", dict(hq=1, hk=1, width=1)),
])
def test_more_work_than_a_launch_holds_is_too_large(name, base, most, change):
    """2^24 workgroups of 256 threads are one thread more than a launch takes; one fewer passes on to the null pointer."""
    each = {128: 16, 64: 32}[change["dim"]] if name == "fp8_kv_append" else 1
    first = {k: None for k in ("k" if name == "fp8_kv_append" else "q",)}
    limit = (2 ** 24 - 1) * each
    assert call(name, base, **change, **first, **{most: limit}) == NULLP
    assert call(name, base, **change, **first, **{most: limit + 1}) == LARGE
    assert call(name, base, **change, **first, **{most: 2 ** 29}) == LARGE


def test_more_work_than_a_launch_holds_by_rows():
    """Paged attention for few rows needs a workgroup for 32, for many one for 128."""
    big = dict(q=None, hq=1, hk=1, tokens=2 ** 29 + 2 ** 20, width=1, max_new=1)
    assert call("fp8_attn_paged", PAGED, **big, batch=2 ** 23 + 2 ** 15) == LARGE     # 64 rows a request at most: for few
    assert call("fp8_attn_paged", PAGED, **big, batch=2 ** 12) == NULLP                # for many


# The plan's buffers apart from each other, 4 KiB each; taken_in and what follows are never dereferenced here.
APART = dict(PLAN, **{n: A + 4096 * i for i, n in enumerate(("cached", "added", "table", "free", "taken", "cu", "lens", "positions",
                                                             "slots", "taken_out", "missing"))})


@pytest.mark.parametrize("out", ["table", "cu", "lens", "positions", "slots", "taken_out", "missing"])
@pytest.mark.parametrize("other", ["cached", "added", "free", "taken", "table", "cu", "lens", "positions", "slots", "taken_out", "missing"])
def test_plan_refuses_outputs_that_share_memory(out, other):
    """Lengths advanced in place (seq_lens is cached) would be read by other workgroups after they are written."""
    if out == other:
        return
    assert call("fp8_paged_plan", APART, **{out: APART[other]}) == SHAPE
    size = dict(cached=16, added=16, table=128, free=20, taken=4, cu=20, lens=16, positions=40, slots=80, taken_out=4, missing=4)[other]
    last = APART[other] + size - 4              # the other's last entry
    if out != "slots" or last % 8 == 0:
        assert call("fp8_paged_plan", APART, **{out: last}) == SHAPE
