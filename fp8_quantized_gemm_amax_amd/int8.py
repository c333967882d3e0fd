"""Python binding of the 8-bit integer product: the C ABI of include/fp8amax_int8.h with the same
names.  Like binding.py: argument marshalling only, and no fallback; compiled with that of the
serving operators (csrc/serving_binding.cpp), since a step's small calls run for a few
microseconds on the GPU."""

import ctypes

import torch

from . import binding, serving
from .binding import _I64, _P

_SIGNATURES = {
    "int8_quantize_rowwise": ([_P, ctypes.c_int, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "int8_gemm_scaled_rowwise": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_int, _P], ctypes.c_int),
}

_fns = None


def _lib():
    """The library's integer functions, bound once (raises if the library has not been built)."""
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


def int8_quantize_rowwise(x, q=None, scales=None):
    """One scale per row, amax * (1 / 127), and the nearest integers (a token of the activations, an
    output channel of the weights).  Returns (q int8 [R, C], scales float32 [R])."""
    r = (serving._ext or serving._load()).quantize8(x, q, scales, serving._stream(x))
    if r.__class__ is int:
        serving._refuse("int8_quantize_rowwise", r)
    return r


def int8_gemm_scaled_rowwise(qa, sa, qb, sb, out_dtype=torch.bfloat16, out=None):
    """C [M, N] = (qa @ qb^T) * sa[m] * sb[n]; qa int8 [M, K], qb int8 [N, K]; sa float32 [M] (per
    token), sb float32 [N] (per output channel).  out_dtype is a new output's; `out` keeps its own type."""
    if out is None:
        binding._out_dt(out_dtype)
    r = (serving._ext or serving._load()).gemm8(qa, sa, qb, sb, out_dtype is torch.bfloat16, out, serving._stream(qa))
    if r.__class__ is int:
        serving._refuse("int8_gemm_scaled_rowwise", r)
    return r
