"""Python binding of the serving operators: the C ABI of include/fp8amax_serving.h with the same
names.

Like binding.py: argument marshalling only, torch supplies device memory and the current
stream, every step runs in the library's HIP kernels, and there is no fallback.  The
marshalling itself is compiled (csrc/serving_binding.cpp): a step's small calls run for a few
microseconds on the GPU, and checking a dozen tensors in Python takes as long.
"""

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple

import torch

from . import binding
from .binding import Fp8Error

FP8_KV_SAME, FP8_KV_E4M3 = 0, 1
COUNTER_BYTES = 16384          # FP8_ATTN_COUNTER_BYTES
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_serving.so")

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
    "fp8_attn_paged": ([_P, ctypes.c_int, _I64, _P, _I64, _I64, _I64, _I32, _I64, _I64, ctypes.c_int, _P, _P, _P, _P,
                        _I64, _I32, _P, _I64, _P, _F32, _I64, _I64, _P, _P, _P, _I64, _P], ctypes.c_int),
    "fp8_attn_paged_workspace": ([_I64, _I64, _I64, _I64, _I32, _I64, _I32, _I64], ctypes.c_int64),
}

_fns = None
_ext = None


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


def _load():
    """The compiled marshalling, loaded once and given the library's addresses."""
    global _ext
    if _ext is None:
        fns = _lib()
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"{BINDING_PATH} is missing: build it with "
                               "`python -m fp8_quantized_gemm_amax_amd.build`")
        loader = importlib.machinery.ExtensionFileLoader("_serving", BINDING_PATH)
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("_serving", loader))
        loader.exec_module(ext)
        ext.bind(*(ctypes.cast(fns[n], _P).value for n in _SIGNATURES))
        _ext = ext
    return _ext


# The current stream's handle of a GPU (torch.cuda.current_stream builds an object around it, at 2 us).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(t):
    """The handle of the current stream on t's GPU; 0 for what the binding is about to refuse."""
    gpu = t.get_device() if isinstance(t, torch.Tensor) else -1
    return _raw_stream(gpu) if gpu >= 0 else 0


def _refuse(name, code):
    raise Fp8Error(name, code, binding.lib().fp8_status_string(code).decode())


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
    ints = torch.empty((2 * batch + tokens + 3,), dtype=torch.int32, device=device)
    cu, lens, positions, taken, missing = ints.split([batch + 1, batch, tokens, 1, 1])
    return PagedPlan(cu, lens, positions, torch.empty((tokens,), dtype=torch.int64, device=device), taken, missing)


def fp8_paged_plan(cached, added, block_table, free_pages, taken, tokens, page_size, out=None):
    """Block tables, slots and positions of one step (see fp8_paged_plan in the header).

    cached, added int32 [batch]; block_table int32 [batch, width], updated in place; free_pages
    int32 [n]; taken int32 [1], how many of them are in use; tokens: the size of the step's token
    buffers.  Returns a PagedPlan; its `taken` is the next step's, `missing` is 0 unless pages
    ran out."""
    r = (_ext or _load()).paged_plan(cached, added, block_table, free_pages, taken, tokens, page_size, out, _stream(cached))
    if r.__class__ is int:
        _refuse("fp8_paged_plan", r)
    return r if out is not None else PagedPlan._make(r)


def fp8_kv_append(k, v, slots, k_cache, v_cache, k_scales=None, v_scales=None):
    """New keys and values [tokens, kv_heads, head_dim] into their slots (int64 [tokens], -1:
    skipped) of the caches [pages, kv_heads, page_size, head_dim], in place: of k's type, or
    e4m3 codes with float32 scales [pages, kv_heads, page_size]."""
    code = (_ext or _load()).kv_append(k, v, slots, k_cache, v_cache, k_scales, v_scales, _stream(k))
    if code:
        _refuse("fp8_kv_append", code)
    return k_cache, v_cache


def fp8_attn_prompt(q, k, v, cu_tokens, softmax_scale=None, window=0, out=None, return_lse=False):
    """Causal attention over whole packed prompts.

    q [tokens, q_heads, head_dim], k and v [tokens, kv_heads, head_dim] (views of a fused
    projection are read in place); cu_tokens int32 [batch + 1].  softmax_scale defaults to
    head_dim ** -0.5; window > 0 limits a query to the last `window` keys.  Returns out
    [tokens, q_heads, head_dim], and with return_lse the float32 [tokens, q_heads] logarithms of
    the softmax sums."""
    r = (_ext or _load()).attn_prompt(q, k, v, cu_tokens, softmax_scale, window, out, return_lse, _stream(q))
    if r.__class__ is int:
        _refuse("fp8_attn_prompt", r)
    return r


def fp8_attn_paged(q, k_cache, v_cache, block_table, seq_lens, cu_tokens, k_scales=None, v_scales=None,
                   softmax_scale=None, window=0, max_new=0, out=None, return_lse=False, workspace=None):
    """Causal attention of each request's new tokens over its pages, the new ones among them.

    q [tokens, q_heads, head_dim] packed by cu_tokens int32 [batch + 1]; caches and scales as
    fp8_kv_append writes them; block_table int32 [batch, width]; seq_lens int32 [batch], tokens in
    the cache.  max_new: the largest number of new tokens of a request if known (it only chooses
    the kernel).  workspace: uint8, at least fp8_attn_paged_workspace(...) bytes, its first
    16 KiB zero before the first call; one per stream is kept by default (a call captured in a HIP
    graph gets one of its own).  Returns as fp8_attn_prompt."""
    r = (_ext or _load()).attn_paged(q, k_cache, v_cache, block_table, seq_lens, cu_tokens, k_scales, v_scales,
                                     softmax_scale, window, max_new, out, return_lse, workspace, _stream(q))
    if r.__class__ is int:
        _refuse("fp8_attn_paged", r)
    return r


def fp8_attn_paged_workspace(tokens, batch, q_heads, kv_heads, head_dim, width, page_size, max_new=0):
    """Bytes of workspace fp8_attn_paged needs for these sizes (0 for sizes it refuses)."""
    return _lib()["fp8_attn_paged_workspace"](tokens, batch, q_heads, kv_heads, head_dim, width, page_size, max_new)
