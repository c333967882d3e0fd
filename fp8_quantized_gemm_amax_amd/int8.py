"""Python binding of the 8-bit integer product: the C ABI of include/fp8amax_int8.h with the same
names.  Like binding.py: argument marshalling only, and no fallback."""

import contextlib
import ctypes

import torch

from . import binding
from .binding import _F32, _I64, _OUT, _P, _as_2d, _check, _check_out, _dt, _need_cuda, _out_dt, _ptr, _same_device, _stream

_I8 = (torch.int8,)
_SIGNATURES = {
    "int8_quantize_rowwise": ([_P, ctypes.c_int, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "int8_gemm_scaled_rowwise": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_int, _P], ctypes.c_int),
}

_fns = None


def _on(device):
    """The launch goes to the tensors' GPU: entered only where that is not the current one."""
    return contextlib.nullcontext() if device.index == torch.cuda.current_device() else torch.cuda.device(device)


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
    """One scale per row, amax / 127, and the nearest integers (a token of the activations, an output
    channel of the weights).  Returns (q int8 [R, C], scales float32 [R])."""
    x = _as_2d(x)
    _need_cuda(x)
    R, C = x.shape
    if q is None:
        q = torch.empty((R, C), dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty((R,), dtype=torch.float32, device=x.device)
    _check_out(q, (R, C), _I8, "q", x, (x,))
    _check_out(scales, (R,), _F32, "scales", x, (x, q))
    with _on(x.device):
        _check("int8_quantize_rowwise",
               _lib()["int8_quantize_rowwise"](_ptr(x), _dt(x), R, C, _ptr(q), _ptr(scales), _stream(x)))
    return q, scales


def int8_gemm_scaled_rowwise(qa, sa, qb, sb, out_dtype=torch.bfloat16, out=None):
    """C [M, N] = (qa @ qb^T) * sa[m] * sb[n]; qa int8 [M, K], qb int8 [N, K]; sa float32 [M] (per
    token), sb float32 [N] (per output channel)."""
    if qa.dtype != torch.int8 or qb.dtype != torch.int8:
        raise TypeError(f"operands must be int8, got {qa.dtype} and {qb.dtype}")
    qa, qb = _as_2d(qa), _as_2d(qb)
    _same_device(qa, qb, sa, sb)
    M, K = qa.shape
    N, K2 = qb.shape
    if K != K2:
        raise ValueError(f"K mismatch: qa has {K}, qb has {K2}")
    if sa.numel() != M or sb.numel() != N:
        raise ValueError(f"scales must have {M} and {N} entries, got {sa.numel()} and {sb.numel()}")
    if sa.dtype != torch.float32 or sb.dtype != torch.float32:
        raise TypeError("scales must be torch.float32")
    sa, sb = sa.contiguous(), sb.contiguous()
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=qa.device)
    _check_out(out, (M, N), _OUT, "out", qa, (qa, qb, sa, sb))
    with _on(qa.device):
        _check("int8_gemm_scaled_rowwise",
               _lib()["int8_gemm_scaled_rowwise"](_ptr(qa), _ptr(sa), _ptr(qb), _ptr(sb), M, N, K, _ptr(out), _out_dt(out.dtype),
                                                  _stream(qa)))
    return out
