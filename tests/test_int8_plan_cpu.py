"""The dispatcher of the 8-bit integer product, on the host (no GPU): the launches of every shape of the
sweep cover the output, and the ranges and offsets that their kernels form in 32 bits stay below 2^31,
also where K is no multiple of 128 and where the operands change places."""

import ctypes
import itertools

import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from fp8_quantized_gemm_amax_amd.binding import lib
from test_gemm_plan_cpu import LIMIT32, MS, NS, cdiv, check_plan, too_large

KS = [16, 112, 128, 144, 1008, 2048, 4096, 4112, 7168, 8192, 8208, 14112, 65536, 131056]
NS8 = sorted(NS + [2, 4, 5, 8, 13])


def plan(M, N, K):
    return fp8.fp8_debug_gemm_plan("int8", M, N, K)


def swaps(M, N):
    """Up to 16 channels for more tokens, as long as a launch holds the threads: fewer than 2^32."""
    return N <= 16 < M and (256 * cdiv(M, 4) if N == 1 else 128 * cdiv(M, 16)) < 2 ** 32


def check(M, N, K, launches):
    swapped = swaps(M, N)
    assert launches[0]["n_begin"] == 0 and launches[-1]["n_end"] == (M if swapped else N)
    for a, b in zip(launches, launches[1:]):
        assert a["n_end"] == b["n_begin"] and a["n_begin"] < a["n_end"]
    m, n = (N, M) if swapped else (M, N)            # as the kernels see them
    if N <= 16 < M < 2 ** 31 - 256:
        assert all(L["grid"] * L["threads"] < 2 ** 32 for L in launches)
    for L in launches:
        kind, cols = L["kernel"], L["n_end"] - L["n_begin"]
        assert L["swapped"] == swapped
        assert 1 <= L["grid"] <= LIMIT32 and L["threads"] == 64 * L["waves"] + (64 if kind == "skinny" else 0)
        assert 0 < L["max_range"] <= LIMIT32 and 0 < L["max_offset"] <= LIMIT32
        tail = 0 if K % 128 == 0 else 128 - K % 128  # past a row's end, up to the last slab's
        if kind == "gemv_valu":
            assert m == 1 and L["grid"] * 4 >= n and L["max_offset"] >= K
        elif kind == "gemv_mfma":
            assert 2 <= m <= 16
            rows = L["tile_n"]
            assert rows == 16 * L["variant"] and L["variant"] == (1 if m <= 4 or swapped else 2) and L["waves"] == 2 * L["variant"]
            assert L["grid"] == cdiv(n, rows)
            assert L["max_offset"] >= rows * K + tail and L["max_range"] >= max(min(rows, n) * K, m * K)
        elif kind == "skinny":
            assert 17 <= m <= 128 and 16 * L["variant"] >= m
            assert L["tile_n"] == 16 * L["waves"] and L["grid"] == cdiv(n, L["tile_n"])
            assert L["max_offset"] >= 16 * L["variant"] * K + tail and L["max_range"] >= max(m, min(16, n)) * K
        else:
            assert kind == "tile" and m > 128
            bm, bn = L["tile_m"], L["tile_n"]
            assert L["grid"] == cdiv(m, bm) * cdiv(cols, bn)
            assert L["paired"] == ((bm, bn) == (256, 256))
            assert L["max_offset"] >= max(bm, bn) * K + tail and L["max_range"] >= max(min(bm, m), min(bn, cols)) * K


def test_every_accepted_shape_has_a_plan_within_32_bit_addressing():
    seen = set()
    for M, N, K in itertools.product(MS, NS8, KS):
        if too_large(M, N, K):
            with pytest.raises(fp8.Fp8Error, match="TOO_LARGE"):
                plan(M, N, K)
            continue
        launches = plan(M, N, K)
        check(M, N, K, launches)
        for L in launches:
            seen.add((L["kernel"], L["swapped"], L["tile_m"] if L["kernel"] == "tile" else 0, L["tile_n"] if L["kernel"] == "tile" else 0, L["variant"]))
    assert {s for s in seen if s[0] != "tile"} == {("gemv_valu", 0, 0, 0, 4), ("gemv_valu", 1, 0, 0, 4), ("gemv_mfma", 0, 0, 0, 1), ("gemv_mfma", 0, 0, 0, 2),
                                                  ("gemv_mfma", 1, 0, 0, 1), ("skinny", 0, 0, 0, 2), ("skinny", 0, 0, 0, 4), ("skinny", 0, 0, 0, 8)}
    assert {s[2:] for s in seen if s[0] == "tile"} == {(256, 256, 2), (256, 128, 2), (256, 128, 3), (128, 128, 2), (128, 128, 3), (128, 96, 3)}


def test_whole_slabs_have_the_launches_of_the_product_with_a_scale_a_row():
    for M, N, K in itertools.product(MS, NS8, [k for k in KS if k % 128 == 0]):
        if not too_large(M, N, K) and not (N <= 16 < M):
            launches = plan(M, N, K)
            check_plan("rowwise", M, N, K, launches)
            assert launches == fp8.fp8_debug_gemm_plan("rowwise", M, N, K)


@pytest.mark.parametrize("N,most", [(1, 2 ** 26 - 4), (2, 2 ** 29 - 16), (16, 2 ** 29 - 16)])
def test_operands_change_places_only_where_a_launch_holds_the_tokens(N, most):
    (a,), (b,) = plan(most, N, 16), plan(most + 1, N, 16)
    assert a["swapped"] and a["kernel"].startswith("gemv") and 2 ** 32 - 256 <= a["grid"] * a["threads"] < 2 ** 32
    assert not b["swapped"] and b["kernel"] == "tile" and b["grid"] * b["threads"] < 2 ** 32


def test_query_errors():
    buffer = ctypes.create_string_buffer(256)
    name = fp8.binding.STATUS_NAMES
    for shape, status in (((-1, 16, 128), "FP8_ERR_BAD_SHAPE"), ((16, 16, 24), "FP8_ERR_BAD_SHAPE"), ((16, 16, 0), "FP8_ERR_BAD_SHAPE"),
                          ((16, 16, 131072), "FP8_ERR_TOO_LARGE"), ((2 ** 31, 16, 16), "FP8_ERR_TOO_LARGE"), ((2 ** 21, 2 ** 20, 16), "FP8_ERR_TOO_LARGE")):
        assert name[lib().fp8_debug_gemm_plan(4, *shape, buffer)] == status, shape
    assert name[lib().fp8_debug_gemm_plan(5, 16, 16, 128, buffer)] == "FP8_ERR_BAD_SHAPE"
    assert plan(0, 16, 128) == [] and plan(16, 0, 128) == [] and plan(100, 0, 128) == []
    with pytest.raises(ValueError, match="mode must be one of"):      # no one-token step in integers
        fp8.fp8_gemv_dynamic("int8", torch.zeros(16, dtype=torch.bfloat16), torch.zeros((4, 16), dtype=torch.uint8), torch.ones(1))
