"""The 8-bit integer entry points, host side (no GPU): what include/fp8amax_int8.h declares is exported
and bound, bad arguments are refused before any HIP call, and the checks of this and of the rotation's
entry point are clean under host sanitizers."""

import os
import re
import subprocess
import sys

import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from fp8_quantized_gemm_amax_amd import binding, build, int8
from test_abi_sanitized_cpu import asan_runtime

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLP, SHAPE, DTYPE, ALIGN, LAUNCH, LARGE = range(7)
A = 0x10000            # fake, aligned addresses (never dereferenced: validation fails first)
QUANT = dict(x=A, dt=0, rows=4, cols=64, q=A, scales=A, stream=None)
GEMM = dict(qa=A, sa=A, qb=A, sb=A, M=4, N=8, K=64, c=A, dt=0, stream=None)


def call(name, base, **change):
    return int8._lib()[name](*dict(base, **change).values())


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "fp8amax_int8.h")).read()
    names = re.findall(r"^fp8_status_t\s+(int8_\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(int8._SIGNATURES) == set(int8._lib())


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(dt=2), DTYPE), (dict(rows=2 ** 31), LARGE), (dict(cols=2 ** 31), LARGE),
    (dict(rows=2 ** 30, cols=2 ** 30), LARGE), (dict(x=None), NULLP), (dict(q=None), NULLP), (dict(scales=None), NULLP),
    (dict(x=A + 2), ALIGN), (dict(q=A + 8), ALIGN), (dict(scales=A + 2), ALIGN), (dict(rows=0, x=None, q=None, scales=None), OK)])
def test_quantize_refusals(change, status):
    assert call("int8_quantize_rowwise", QUANT, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=-16), SHAPE), (dict(K=24), SHAPE), (dict(K=131072), LARGE),
    (dict(K=2 ** 40), LARGE), (dict(M=2 ** 31), LARGE), (dict(N=2 ** 31), LARGE), (dict(M=2 ** 28, N=2 ** 28), LARGE), (dict(dt=2), DTYPE),
    (dict(qa=None), NULLP), (dict(sa=None), NULLP), (dict(qb=None), NULLP), (dict(sb=None), NULLP), (dict(c=None), NULLP),
    (dict(qa=A + 8), ALIGN), (dict(qb=A + 1), ALIGN), (dict(c=A + 4), ALIGN), (dict(sa=A + 2), ALIGN), (dict(sb=A + 1), ALIGN),
    (dict(M=0, qa=None, c=None), OK), (dict(N=0), OK)])
def test_gemm_refusals(change, status):
    assert call("int8_gemm_scaled_rowwise", GEMM, **change) == status


def codes(*shape):
    return torch.zeros(shape, dtype=torch.int8)


T, V = TypeError, ValueError


@pytest.mark.parametrize("error,match,f", [
    (V, "2-D", lambda: fp8.int8_quantize_rowwise(torch.zeros(4, dtype=torch.bfloat16))),
    (V, "on the GPU", lambda: fp8.int8_quantize_rowwise(torch.zeros((4, 8), dtype=torch.bfloat16))),
    (T, "must be int8", lambda: fp8.int8_gemm_scaled_rowwise(codes(4, 16).view(torch.uint8), torch.ones(4), codes(8, 16), torch.ones(8))),
    (T, "must be int8", lambda: fp8.int8_gemm_scaled_rowwise(codes(4, 16), torch.ones(4), codes(8, 16).float(), torch.ones(8))),
    (V, "2-D", lambda: fp8.int8_gemm_scaled_rowwise(codes(16), torch.ones(4), codes(8, 16), torch.ones(8))),
    (V, "on the GPU", lambda: fp8.int8_gemm_scaled_rowwise(codes(4, 16), torch.ones(4), codes(8, 16), torch.ones(8))),
])
def test_binding_refuses(error, match, f):
    with pytest.raises(error, match=match):
        f()


def test_checks_clean_under_host_sanitizers(tmp_path):
    rt = asan_runtime()
    apis = ("api.hip", "serving_api.hip")
    objs = [os.path.join(build.OBJ_DIR, s.replace(".hip", ".o")) for s in build.SOURCES if s not in apis]
    if rt is None or not all(os.path.exists(o) for o in objs):
        pytest.skip("no sanitizer runtime, or the library has not been built")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all"]
    flags = [f for f in build.HIPCC_FLAGS if f != "-O3"] + ["-O1", "-g"]
    cc, lib = build.hipcc(), str(tmp_path / "libfp8amax_san.so")
    for s in apis:
        subprocess.run([cc, *flags, *san, "-shared-libasan", "-I", build.INCLUDE, "-I", build.CSRC, "-c", "-o", str(tmp_path / (s + ".o")),
                        os.path.join(build.CSRC, s)], check=True, capture_output=True, timeout=600)
    subprocess.run([cc, "--offload-arch=gfx950", "-shared", "-fPIC", *san, "-shared-libasan", "-o", lib, *(str(tmp_path / (s + ".o")) for s in apis), *objs],
                   check=True, capture_output=True, timeout=600)
    env = dict(os.environ, FP8AMAX_LIBRARY=lib, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-s", "-p", "no:cacheprovider", "-m", "not gpu", "-k", "not binding and not sanitizers and not table",
                        "tests/test_int8_abi_cpu.py", "tests/test_rope_abi_cpu.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in r.stdout
