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


def _refuse(name, code):
    raise Fp8Error(name, code, binding.lib().fp8_status_string(code).decode())


# The current stream's handle of a GPU; torch.cuda.current_stream builds an object around it, which
# takes 1.8 of the 8 to 11 us that a call takes on the host.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _on(like, **tensors):
    """Every given tensor is a tensor on like's GPU (the library launches on like's stream)."""
    if not like.is_cuda:
        raise ValueError("all tensors must be on the GPU")
    for what, t in tensors.items():
        if t.device != like.device:
            raise ValueError(f"{what} must be on {like.device}, got {t.device}")


def _dense(t, what, dtype, shape):
    """A dense operand of one type and shape, read or written where it lies."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _rows(t, what, head_dim=None):
    """A [tokens, heads, dim] operand whose rows the kernels read 16 bytes at a time: as it lies
    if its last index is contiguous, the other strides are multiples of 8 and tokens do not overlap,
    else a copy.  Returns the tensor, its address and its token and head strides."""
    if t.dim() != 3:
        raise ValueError(f"{what} must be [tokens, heads, head_dim], got shape {tuple(t.shape)}")
    if head_dim is not None and t.shape[2] != head_dim:
        raise ValueError(f"{what} must have head_dim {head_dim}, got {t.shape[2]}")
    ts, hs, one = t.stride()
    at = t.data_ptr()
    if one != 1 or (ts | hs | at >> 1) & 7 or ts < t.shape[2] or ts > 1 << 20:
        t = t.contiguous()
        if t.data_ptr() & 15:
            t = t.clone()
        ts, hs, _ = t.stride()
        at = t.data_ptr()
    return t, at, ts, hs


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
    return _plan_buffers(torch.empty((3 * tokens + 2 * batch + 3,), dtype=torch.int32, device=device), batch, tokens)


def _plan_buffers(ints, batch, tokens):
    # one allocation, the 64-bit slots first
    slots, positions, cu, lens, taken, missing = ints.unsafe_split_with_sizes([2 * tokens, tokens, batch + 1, batch, 1, 1])
    return PagedPlan(cu, lens, positions, slots.view(torch.int64), taken, missing)


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
    gpu = cached.get_device()
    if gpu < 0 or not gpu == added.get_device() == block_table.get_device() == free_pages.get_device() == taken.get_device():
        _on(cached, added=added, block_table=block_table, free_pages=free_pages, taken=taken)
    if out is None:
        if tokens < 0:
            raise ValueError(f"tokens must not be negative, got {tokens}")
        ints = cached.new_empty(3 * tokens + 2 * batch + 3)
        out = _plan_buffers(ints, batch, tokens)
        # the parts' addresses, in paged_plan_buffers' order
        slots = ints.data_ptr()
        positions = slots + 8 * tokens
        cu = positions + 4 * tokens
        lens = cu + 4 * (batch + 1)
        taken_out = lens + 4 * batch
        missing = taken_out + 4
    else:
        for what, dtype, n in (("cu_tokens", torch.int32, batch + 1), ("seq_lens", torch.int32, batch),
                               ("positions", torch.int32, tokens), ("slots", torch.int64, tokens),
                               ("taken", torch.int32, 1), ("missing", torch.int32, 1)):
            t = getattr(out, what)
            binding._check_out(t, (n,), (dtype,), f"out.{what}", cached, (cached, added, block_table, free_pages, taken))
        cu, lens, positions, slots, taken_out, missing = (t.data_ptr() for t in out)
    code = (_fns or _lib())["fp8_paged_plan"](
        cached.data_ptr(), added.data_ptr(), batch, page_size, block_table.data_ptr(), block_table.shape[1],
        free_pages.data_ptr(), free_pages.shape[0], taken.data_ptr(), tokens, cu, lens, positions, slots, taken_out,
        missing, _raw_stream(gpu))
    if code:
        _refuse("fp8_paged_plan", code)
    return out


def _cache(k_cache, v_cache, k_scales, v_scales, dtype):
    """Shape (pages, heads, page_size, dim) and format of a cache."""
    shape, kind = k_cache.shape, k_cache.dtype
    if len(shape) != 4:
        raise ValueError(f"k_cache must be [pages, kv_heads, page_size, head_dim], got {tuple(shape)}")
    if v_cache.dtype != kind:
        raise TypeError(f"k_cache and v_cache must have one type, got {kind} and {v_cache.dtype}")
    _dense(k_cache, "k_cache", kind, shape)
    _dense(v_cache, "v_cache", kind, shape)
    if (k_scales is None) != (v_scales is None):
        raise ValueError("k_scales and v_scales go together")
    if k_scales is None:
        if kind != dtype:
            raise TypeError(f"a cache without scales must be {dtype}, got {kind}")
        return shape, FP8_KV_SAME
    if kind not in _CODE_TYPES:
        raise TypeError(f"a cache with scales must be uint8 or float8_e4m3fn, got {kind}")
    _dense(k_scales, "k_scales", torch.float32, shape[:3])
    _dense(v_scales, "v_scales", torch.float32, shape[:3])
    return shape, FP8_KV_E4M3


def fp8_kv_append(k, v, slots, k_cache, v_cache, k_scales=None, v_scales=None):
    """New keys and values [tokens, kv_heads, head_dim] into their slots (int64 [tokens], -1:
    skipped) of the caches [pages, kv_heads, page_size, head_dim], in place: of k's type, or
    e4m3 codes with float32 scales [pages, kv_heads, page_size]."""
    dt = _dt(k, "k")
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError(f"v must be like k, got {v.dtype} {tuple(v.shape)} and {k.dtype} {tuple(k.shape)}")
    (pages, heads, page, dim), fmt = _cache(k_cache, v_cache, k_scales, v_scales, k.dtype)
    k, k_at, kts, khs = _rows(k, "k", dim)
    v, v_at, vts, vhs = _rows(v, "v", dim)
    tokens = k.shape[0]
    if k.shape[1] != heads:
        raise ValueError(f"k has {k.shape[1]} heads, the cache {heads}")
    slots = _vector(slots, "slots", torch.int64, tokens)
    gpu = k.get_device()
    if gpu < 0 or not gpu == v.get_device() == slots.get_device() == k_cache.get_device() == v_cache.get_device():
        _on(k, v=v, slots=slots, k_cache=k_cache, v_cache=v_cache)
    ks = vs = None
    if fmt == FP8_KV_E4M3:
        if not gpu == k_scales.get_device() == v_scales.get_device():
            _on(k, k_scales=k_scales, v_scales=v_scales)
        ks, vs = k_scales.data_ptr(), v_scales.data_ptr()
    code = (_fns or _lib())["fp8_kv_append"](
        k_at, v_at, dt, tokens, heads, dim, kts, khs, vts, vhs, slots.data_ptr(), pages, page, fmt,
        k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, _raw_stream(gpu))
    if code:
        _refuse("fp8_kv_append", code)
    return k_cache, v_cache


def _output(q, out, inputs):
    if out is None:
        return torch.empty_like(q) if q.is_contiguous() else q.new_empty(q.shape)
    return binding._check_out(out, tuple(q.shape), (q.dtype,), "out", q, [_span_of(t) for t in inputs if t is not None])


def _sums(q, return_lse):
    return torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if return_lse else None


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
    q, q_at, qts, qhs = _rows(q, "q")
    tokens, hq, dim = q.shape
    k, k_at, kts, khs = _rows(k, "k", dim)
    v, v_at, vts, vhs = _rows(v, "v", dim)
    if k.shape[0] != tokens:
        raise ValueError(f"q has {tokens} tokens, k {k.shape[0]}")
    cu_tokens = _vector(cu_tokens, "cu_tokens")
    gpu = q.get_device()
    if gpu < 0 or not gpu == k.get_device() == v.get_device() == cu_tokens.get_device():
        _on(q, k=k, v=v, cu_tokens=cu_tokens)
    out = _output(q, out, (q, k, v, cu_tokens))
    lse = _sums(q, return_lse)
    code = (_fns or _lib())["fp8_attn_prompt"](
        q_at, k_at, v_at, dt, tokens, cu_tokens.data_ptr(), cu_tokens.shape[0] - 1, hq, k.shape[1], dim, qts, qhs, kts,
        khs, vts, vhs, _scale(softmax_scale, dim), window, out.data_ptr(), lse.data_ptr() if return_lse else None,
        _raw_stream(gpu))
    if code:
        _refuse("fp8_attn_prompt", code)
    return (out, lse) if return_lse else out


_workspaces = {}


def _workspace(q, stream, need):
    """A workspace of the current stream, its counters zero at first and kept: a call leaves it fit
    for the next.  A call that is being captured in a HIP graph gets its own, since the graph may
    be replayed on any stream."""
    capturing = torch.cuda.is_current_stream_capturing()
    key = q.get_device(), stream
    have = None if capturing else _workspaces.get(key)
    if have is None or have.shape[0] < need:
        have = torch.empty((max(need, COUNTER_BYTES),), dtype=torch.uint8, device=q.device)
        have[:COUNTER_BYTES].zero_()
        if not capturing:
            _workspaces[key] = have
    return have


def _check_workspace(q, workspace):
    if workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 vector")
    _on(q, workspace=workspace)


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
    q, q_at, qts, qhs = _rows(q, "q", dim)
    tokens, hq, _ = q.shape
    seq_lens = _vector(seq_lens, "seq_lens")
    batch = seq_lens.shape[0]
    cu_tokens = _vector(cu_tokens, "cu_tokens", size=batch + 1)
    width = _table(block_table, batch).shape[1]
    gpu = q.get_device()
    if gpu < 0 or not gpu == k_cache.get_device() == v_cache.get_device() == block_table.get_device() == seq_lens.get_device() == cu_tokens.get_device():
        _on(q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, seq_lens=seq_lens, cu_tokens=cu_tokens)
    ks = vs = None
    if fmt == FP8_KV_E4M3:
        if not gpu == k_scales.get_device() == v_scales.get_device():
            _on(q, k_scales=k_scales, v_scales=v_scales)
        ks, vs = k_scales.data_ptr(), v_scales.data_ptr()
    out = _output(q, out, (q, k_cache, v_cache, block_table, seq_lens, cu_tokens, k_scales, v_scales))
    lse = _sums(q, return_lse)
    fns = _fns or _lib()
    stream = _raw_stream(gpu)
    if workspace is None:
        workspace = _workspace(q, stream, fns["fp8_attn_paged_workspace"](tokens, batch, hq, hk, dim, width, page, max_new))
    else:
        _check_workspace(q, workspace)
    code = fns["fp8_attn_paged"](
        q_at, dt, tokens, cu_tokens.data_ptr(), batch, hq, hk, dim, qts, qhs, fmt, k_cache.data_ptr(),
        v_cache.data_ptr(), ks, vs, pages, page, block_table.data_ptr(), width, seq_lens.data_ptr(),
        _scale(softmax_scale, dim), window, max_new, out.data_ptr(), lse.data_ptr() if return_lse else None,
        workspace.data_ptr(), workspace.shape[0], stream)
    if code:
        _refuse("fp8_attn_paged", code)
    return (out, lse) if return_lse else out


def fp8_attn_paged_workspace(tokens, batch, q_heads, kv_heads, head_dim, width, page_size, max_new=0):
    """Bytes of workspace fp8_attn_paged needs for these sizes (0 for sizes it refuses)."""
    return _lib()["fp8_attn_paged_workspace"](tokens, batch, q_heads, kv_heads, head_dim, width, page_size, max_new)
