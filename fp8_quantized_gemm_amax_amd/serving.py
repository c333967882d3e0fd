"""ctypes binding of the serving operators: the C ABI of include/fp8amax_serving.h with the
same names.

Like binding.py: argument marshalling only, torch supplies device memory and the current
stream, every step runs in the library's HIP kernels, and there is no fallback.
"""

import ctypes
import math
from typing import NamedTuple

import torch

from . import binding
from .binding import FP8_BF16, FP8_F16, Fp8Error

FP8_KV_SAME, FP8_KV_E4M3 = 0, 1
COUNTER_BYTES = 16384          # FP8_ATTN_COUNTER_BYTES

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_F32 = ctypes.c_float
_SIGNATURES = {
    "fp8_paged_plan": ([_P, _P, _I64, _I32, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "fp8_kv_append": ([_P, _P, ctypes.c_int, _I64, _I64, _I32, _I64, _I64, _I64, _I64, _P, _I64, _I32, ctypes.c_int,
                       _P, _P, _P, _P, _P], ctypes.c_int),
    "fp8_attn_prompt": ([_P, _P, _P, ctypes.c_int, _I64, _P, _I64, _I64, _I64, _I32, _I64, _I64, _I64, _I64, _I64,
                         _I64, _F32, _I64, _P, _P, _P], ctypes.c_int),
    "fp8_attn_paged_workspace": ([_I64, _I64, _I64, _I64, _I32, _I64, _I32, _I64], ctypes.c_int64),
    "fp8_attn_paged": ([_P, ctypes.c_int, _I64, _P, _I64, _I64, _I64, _I32, _I64, _I64, ctypes.c_int, _P, _P, _P, _P,
                        _I64, _I32, _P, _I64, _P, _F32, _I64, _I64, _P, _P, _P, _I64, _P], ctypes.c_int),
}

_fns = None


def _lib():
    """The library's serving functions, bound once (raises if the library has not been built)."""
    global _fns
    if _fns is None:
        handle = binding.lib()
        found = {}
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
            found[name] = fn
        _fns = found
    return _fns


_DT = {torch.bfloat16: FP8_BF16, torch.float16: FP8_F16}
_CODE_TYPES = (torch.uint8, torch.float8_e4m3fn)


def _dt(t, what):
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what} must be bfloat16 or float16, got {t.dtype}")
    return dt


def _check(name, code):
    if code:
        raise Fp8Error(name, code, binding.lib().fp8_status_string(code).decode())


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _on(like, **tensors):
    """Every given tensor is a tensor on like's GPU (the library launches on like's stream)."""
    device = like.device
    if device.type != "cuda":
        raise ValueError("all tensors must be on the GPU")
    for what, t in tensors.items():
        if t.device != device:
            raise ValueError(f"{what} must be on {device}, got {t.device}")


def _dense(t, what, dtype, shape):
    """A dense operand of one type and shape, read or written where it lies."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{what} must have shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _rows(t, what, heads_dim=None):
    """A [tokens, heads, dim] operand whose rows the kernels read 16 bytes at a time: as it lies
    if its last index is contiguous, the other strides are multiples of 8 and tokens do not overlap,
    else a copy."""
    if t.dim() != 3:
        raise ValueError(f"{what} must be [tokens, heads, head_dim], got shape {tuple(t.shape)}")
    if heads_dim is not None and t.shape[2] != heads_dim:
        raise ValueError(f"{what} must have head_dim {heads_dim}, got {t.shape[2]}")
    ts, hs, one = t.stride()
    if one != 1 or (ts | hs) & 7 or t.data_ptr() & 15 or ts < t.shape[2] or ts > 1 << 20:
        t = t.contiguous()
        if t.data_ptr() & 15:
            t = t.clone()
    return t


def _vector(t, what, dtype=torch.int32, size=None):
    if t.dtype != dtype or t.dim() != 1 or (size is not None and t.shape[0] != size):
        raise TypeError(f"{what} must be {dtype} [{'n' if size is None else size}], got {t.dtype} {tuple(t.shape)}")
    return t if t.is_contiguous() else t.contiguous()


def _table(t, batch):
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != batch or not t.is_contiguous():
        raise ValueError(f"block_table must be a contiguous int32 [{batch}, width], got {t.dtype} {tuple(t.shape)}")
    return t


class PagedPlan(NamedTuple):
    """What fp8_paged_plan writes, beside the block table."""
    cu_tokens: torch.Tensor    # int32 [batch + 1]
    seq_lens: torch.Tensor     # int32 [batch]
    positions: torch.Tensor    # int32 [tokens]
    slots: torch.Tensor        # int64 [tokens]
    taken: torch.Tensor        # int32 [1]
    missing: torch.Tensor      # int32 [1]


def paged_plan_buffers(batch, tokens, device):
    """Buffers for fp8_paged_plan's `out` (to reuse them, or to capture the call in a HIP graph)."""
    # one allocation: the int64 slots first, then the int32 outputs
    ints = torch.empty((2 * tokens + 2 * batch + 1 + tokens + 2,), dtype=torch.int32, device=device)
    slots = ints[: 2 * tokens].view(torch.int64)
    positions, cu, lens, taken, missing = ints[2 * tokens:].split([tokens, batch + 1, batch, 1, 1])
    return PagedPlan(cu, lens, positions, slots, taken, missing)


def fp8_paged_plan(cached, added, block_table, free_pages, taken, tokens, page_size, out=None):
    """Block tables, slots and positions of one step (see fp8_paged_plan in the header).

    cached, added int32 [batch]; block_table int32 [batch, width], updated in place; free_pages
    int32 [n]; taken int32 [1], how many of them are in use; tokens: the size of the step's token
    buffers.  Returns a PagedPlan; its `taken` is the next step's, `missing` is 0 unless pages
    ran out."""
    batch = cached.shape[0]
    cached, added = _vector(cached, "cached"), _vector(added, "added", size=batch)
    free_pages, taken = _vector(free_pages, "free_pages"), _vector(taken, "taken", size=1)
    _table(block_table, batch)
    _on(cached, added=added, block_table=block_table, free_pages=free_pages, taken=taken)
    if out is None:
        if tokens < 0:
            raise ValueError(f"tokens must not be negative, got {tokens}")
        out = paged_plan_buffers(batch, tokens, cached.device)
    else:
        for what, dtype, n in (("cu_tokens", torch.int32, batch + 1), ("seq_lens", torch.int32, batch),
                               ("positions", torch.int32, tokens), ("slots", torch.int64, tokens),
                               ("taken", torch.int32, 1), ("missing", torch.int32, 1)):
            t = getattr(out, what)
            binding._check_out(t, (n,), (dtype,), f"out.{what}", cached, (cached, added, block_table, free_pages, taken))
    _check("fp8_paged_plan", _lib()["fp8_paged_plan"](
        cached.data_ptr(), added.data_ptr(), batch, page_size, block_table.data_ptr(), block_table.shape[1],
        free_pages.data_ptr(), free_pages.shape[0], taken.data_ptr(), tokens, out.cu_tokens.data_ptr(),
        out.seq_lens.data_ptr(), out.positions.data_ptr(), out.slots.data_ptr(), out.taken.data_ptr(),
        out.missing.data_ptr(), _stream(cached.device)))
    return out


def _cache(k_cache, v_cache, k_scales, v_scales, dtype, what="k_cache"):
    """Shape (pages, heads, page_size, dim) and format of a cache."""
    if k_cache.dim() != 4:
        raise ValueError(f"{what} must be [pages, kv_heads, page_size, head_dim], got {tuple(k_cache.shape)}")
    shape = tuple(k_cache.shape)
    if v_cache.dtype != k_cache.dtype:
        raise TypeError(f"k_cache and v_cache must have one type, got {k_cache.dtype} and {v_cache.dtype}")
    _dense(k_cache, "k_cache", k_cache.dtype, shape)
    _dense(v_cache, "v_cache", k_cache.dtype, shape)
    if (k_scales is None) != (v_scales is None):
        raise ValueError("k_scales and v_scales go together")
    if k_scales is None:
        if k_cache.dtype != dtype:
            raise TypeError(f"a cache without scales must be {dtype}, got {k_cache.dtype}")
        return shape, FP8_KV_SAME
    if k_cache.dtype not in _CODE_TYPES:
        raise TypeError(f"a cache with scales must be uint8 or float8_e4m3fn, got {k_cache.dtype}")
    _dense(k_scales, "k_scales", torch.float32, shape[:3])
    _dense(v_scales, "v_scales", torch.float32, shape[:3])
    return shape, FP8_KV_E4M3


def _at(t):
    return None if t is None else t.data_ptr()


def fp8_kv_append(k, v, slots, k_cache, v_cache, k_scales=None, v_scales=None):
    """New keys and values [tokens, kv_heads, head_dim] into their slots (int64 [tokens], -1:
    skipped) of the caches [pages, kv_heads, page_size, head_dim], in place: of k's type, or
    e4m3 codes with float32 scales [pages, kv_heads, page_size]."""
    dt = _dt(k, "k")
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError(f"v must be like k, got {v.dtype} {tuple(v.shape)} and {k.dtype} {tuple(k.shape)}")
    (pages, heads, page, dim), fmt = _cache(k_cache, v_cache, k_scales, v_scales, k.dtype)
    k, v = _rows(k, "k", dim), _rows(v, "v", dim)
    if k.shape[1] != heads:
        raise ValueError(f"k has {k.shape[1]} heads, the cache {heads}")
    tokens = k.shape[0]
    slots = _vector(slots, "slots", torch.int64, tokens)
    _on(k, v=v, slots=slots, k_cache=k_cache, v_cache=v_cache)
    if fmt == FP8_KV_E4M3:
        _on(k, k_scales=k_scales, v_scales=v_scales)
    _check("fp8_kv_append", _lib()["fp8_kv_append"](
        k.data_ptr(), v.data_ptr(), dt, tokens, heads, dim, k.stride(0), k.stride(1), v.stride(0), v.stride(1),
        slots.data_ptr(), pages, page, fmt, k_cache.data_ptr(), v_cache.data_ptr(), _at(k_scales), _at(v_scales),
        _stream(k.device)))
    return k_cache, v_cache


def _outputs(q, out, return_lse, inputs):
    shape = tuple(q.shape)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    else:
        binding._check_out(out, shape, (q.dtype,), "out", q, inputs)
    return out, torch.empty(shape[:2], dtype=torch.float32, device=q.device) if return_lse else None


def _scale(softmax_scale, dim):
    return 1.0 / math.sqrt(dim) if softmax_scale is None else softmax_scale


def _span_of(t):
    """A contiguous stand-in covering the memory of a strided operand, for the overlap check."""
    if t.is_contiguous() or t.numel() == 0:
        return t
    n = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride()))
    return t.as_strided((n,), (1,))


def fp8_attn_prompt(q, k, v, cu_tokens, softmax_scale=None, window=0, out=None, return_lse=False):
    """Causal attention over whole packed prompts.

    q [tokens, q_heads, head_dim], k and v [tokens, kv_heads, head_dim] (views of a fused
    projection are read in place); cu_tokens int32 [batch + 1].  softmax_scale defaults to
    head_dim ** -0.5; window > 0 limits a query to the last `window` keys.  Returns out
    [tokens, q_heads, head_dim], and with return_lse the float32 [tokens, q_heads] logarithms of
    the softmax sums."""
    dt = _dt(q, "q")
    if k.dtype != q.dtype or v.dtype != q.dtype or v.shape != k.shape:
        raise ValueError(f"k and v must be alike and of q's type, got {k.dtype} {tuple(k.shape)} and {v.dtype} {tuple(v.shape)}")
    q = _rows(q, "q")
    tokens, hq, dim = q.shape
    k, v = _rows(k, "k", dim), _rows(v, "v", dim)
    if k.shape[0] != tokens:
        raise ValueError(f"q has {tokens} tokens, k {k.shape[0]}")
    cu_tokens = _vector(cu_tokens, "cu_tokens")
    _on(q, k=k, v=v, cu_tokens=cu_tokens)
    out, lse = _outputs(q, out, return_lse, () if out is None else (_span_of(q), _span_of(k), _span_of(v), cu_tokens))
    _check("fp8_attn_prompt", _lib()["fp8_attn_prompt"](
        q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, tokens, cu_tokens.data_ptr(), cu_tokens.shape[0] - 1, hq,
        k.shape[1], dim, q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
        _scale(softmax_scale, dim), window, out.data_ptr(), _at(lse), _stream(q.device)))
    return (out, lse) if return_lse else out


_workspaces = {}


def _workspace(device, need):
    """A workspace of the current stream, its counters zero at first and kept: a call leaves it fit
    for the next.  A call that is being captured in a HIP graph gets its own, since the graph may
    be replayed on any stream."""
    capturing = torch.cuda.is_current_stream_capturing()
    key = device.index, _stream(device)
    have = None if capturing else _workspaces.get(key)
    if have is None or have.shape[0] < need:
        have = torch.empty((need,), dtype=torch.uint8, device=device)
        have[:COUNTER_BYTES].zero_()
        if not capturing:
            _workspaces[key] = have
    return have


def fp8_attn_paged(q, k_cache, v_cache, block_table, seq_lens, cu_tokens, k_scales=None, v_scales=None,
                   softmax_scale=None, window=0, max_new=0, out=None, return_lse=False, workspace=None):
    """Causal attention of each request's new tokens over its pages, the new ones among them.

    q [tokens, q_heads, head_dim] packed by cu_tokens int32 [batch + 1]; caches and scales as
    fp8_kv_append writes them; block_table int32 [batch, width]; seq_lens int32 [batch], tokens in
    the cache.  max_new: the largest number of new tokens of a request if known (it only chooses
    the kernel).  workspace: uint8, at least fp8_attn_paged_workspace(...) bytes, its first
    16 KiB zero before the first call; one per stream is kept by default.  Returns as fp8_attn_prompt."""
    dt = _dt(q, "q")
    (pages, hk, page, dim), fmt = _cache(k_cache, v_cache, k_scales, v_scales, q.dtype)
    q = _rows(q, "q", dim)
    tokens, hq, _ = q.shape
    seq_lens = _vector(seq_lens, "seq_lens")
    batch = seq_lens.shape[0]
    cu_tokens = _vector(cu_tokens, "cu_tokens", size=batch + 1)
    width = _table(block_table, batch).shape[1]
    _on(q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, seq_lens=seq_lens, cu_tokens=cu_tokens)
    if fmt == FP8_KV_E4M3:
        _on(q, k_scales=k_scales, v_scales=v_scales)
    out, lse = _outputs(q, out, return_lse, () if out is None else (
        _span_of(q), k_cache, v_cache, block_table, seq_lens, cu_tokens, k_scales, v_scales))
    fns = _lib()
    need = fns["fp8_attn_paged_workspace"](tokens, batch, hq, hk, dim, width, page, max_new)
    if workspace is None:
        workspace = _workspace(q.device, need) if need else None
    else:
        if workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous uint8 vector")
        _on(q, workspace=workspace)
    _check("fp8_attn_paged", fns["fp8_attn_paged"](
        q.data_ptr(), dt, tokens, cu_tokens.data_ptr(), batch, hq, hk, dim, q.stride(0), q.stride(1), fmt,
        k_cache.data_ptr(), v_cache.data_ptr(), _at(k_scales), _at(v_scales), pages, page, block_table.data_ptr(),
        width, seq_lens.data_ptr(), _scale(softmax_scale, dim), window, max_new, out.data_ptr(), _at(lse),
        _at(workspace), 0 if workspace is None else workspace.shape[0], _stream(q.device)))
    return (out, lse) if return_lse else out


def fp8_attn_paged_workspace(tokens, batch, q_heads, kv_heads, head_dim, width, page_size, max_new=0):
    """Bytes of workspace fp8_attn_paged needs for these sizes (0 for sizes it refuses)."""
    return _lib()["fp8_attn_paged_workspace"](tokens, batch, q_heads, kv_heads, head_dim, width, page_size, max_new)
