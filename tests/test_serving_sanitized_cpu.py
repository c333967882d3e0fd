"""The serving operators' host-side argument checks under AddressSanitizer and
UndefinedBehaviorSanitizer (no GPU): serving_api.hip is rebuilt with the sanitizers on its host
code only, linked with the other objects of the normal build, and the host-side tests run
against that library in a child process with the sanitizer runtime preloaded."""

import os
import subprocess
import sys

import pytest

from fp8_quantized_gemm_amax_amd import build
from test_abi_sanitized_cpu import asan_runtime

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_serving_checks_clean_under_host_sanitizers(tmp_path):
    rt = asan_runtime()
    objs = [os.path.join(build.OBJ_DIR, s.replace(".hip", ".o")) for s in build.SOURCES if s != "serving_api.hip"]
    if rt is None or not all(os.path.exists(o) for o in objs):
        pytest.skip("no sanitizer runtime, or the library has not been built")
    # sanitizers on the host pass only: -Xarch_host right before each option
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all"]
    flags = [f for f in build.HIPCC_FLAGS if f != "-O3"] + ["-O1", "-g"]
    api_o, lib = str(tmp_path / "serving_api_san.o"), str(tmp_path / "libfp8amax_san.so")
    cc = build.hipcc()
    subprocess.run([cc, *flags, *san, "-shared-libasan", "-I", build.INCLUDE, "-I", build.CSRC, "-c", "-o", api_o,
                    os.path.join(build.CSRC, "serving_api.hip")], check=True, capture_output=True, timeout=600)
    subprocess.run([cc, "--offload-arch=gfx950", "-shared", "-fPIC", *san, "-shared-libasan", "-o", lib, api_o, *objs],
                   check=True, capture_output=True, timeout=600)
    env = dict(os.environ, FP8AMAX_LIBRARY=lib, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    # the binding's own C++ exceptions need the runtime's interceptors and are not what is tested here
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-s", "-p", "no:cacheprovider", "-m", "not gpu", "-k", "not binding",
                        "tests/test_serving_abi_cpu.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in r.stdout
