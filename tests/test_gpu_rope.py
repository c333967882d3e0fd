"""Rotation with append: the queries and the cache bit for bit what float32 products and sums, rounded
once, give; sizes, strides, positions and slots where it can go wrong; and a step of the operators as
they are used together, eager, on another stream and in a graph."""

import math

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from mxfp4_util import Cache4
from oracle import decode_e4m3, encode_e4m3, mxfp4
from parity_util import DEV
from serving_util import TORCH, bits_of, check_paged, cu_of, f64_of, normal

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def stored(x, dtype, fmt):
    """What a cache of the format holds for float32 rows x [..., D]: (codes or bits, scales)."""
    if fmt == "same":
        return bits_of(torch.from_numpy(x).to(TORCH[dtype])), None
    if fmt == "mxfp4":
        return mxfp4.quantize(x, dtype)
    amax = np.where(np.isnan(x).any(-1), np.float32(np.nan), np.abs(x).max(-1)).astype(np.float32)
    scale = np.where(amax == 0, np.float32(1), amax / np.float32(448)).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        return encode_e4m3((x / scale[..., None]).astype(np.float32)), scale


def run_rope(tokens, hq, hk, dim, rotary, page, dtype, fmt, interleaved, seed=0, special=True):
    rng = np.random.default_rng(seed + tokens)
    fused = normal((tokens, hq + 2 * hk + 1, dim), dtype, seed + tokens, 2.0)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk + 1:]
    table = fp8.rope_table(300, rotary, device=DEV)
    positions = rng.integers(0, 300, tokens).astype(np.int32)
    pages = -(-tokens // page) + 2
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 8 and special:
        positions[0], positions[-1], positions[3] = -1, 300, -(1 << 31)          # skipped tokens
        slots[1], slots[2], slots[-2] = -1, pages * page, 1 << 40                # queries only
        k[4], v[4] = 0.0, 0.0
        k[5, 0, 3], v[5, 0, 3], q[5, 0, 1] = float("nan"), float("nan"), float("inf")
        v[6, 0, 7] = float("inf")
        k[7] = torch.finfo(TORCH[dtype]).max * 0.6
        v[7] *= 2.0 ** -15
    width = {"same": dim, "e4m3": dim, "mxfp4": dim // 2}[fmt]
    kind = TORCH[dtype] if fmt == "same" else torch.uint8
    caches = [torch.full((pages, hk, page, width), 9, dtype=kind, device=DEV) for _ in "kv"]
    scales = [None, None]
    if fmt != "same":
        scales = [torch.full((pages, hk, page) + (() if fmt == "e4m3" else (dim // 32,)), 77, dtype=torch.float32 if fmt == "e4m3" else torch.uint8, device=DEV) for _ in "kv"]
    full = torch.full((tokens * hq * dim + 512,), -7.0, dtype=TORCH[dtype], device=DEV)
    out = full[: tokens * hq * dim].view(tokens, hq, dim)
    got = fp8.fp8_rope_append(q if hq else None, k, v, i32(positions), table, torch.from_numpy(slots).to(DEV), *caches, *scales, interleaved=interleaved,
                              out=out if hq else None)
    torch.cuda.synchronize()
    assert (got is out) if hq else got is None
    assert (full[tokens * hq * dim:] == -7.0).all()
    there = (positions >= 0) & (positions < 300)
    at, tab = np.where(there, positions, 0), table.cpu().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        if hq:
            want = torch.from_numpy(mxfp4.rotate(q.float().cpu().numpy(), at, tab, interleaved)).to(TORCH[dtype])
            want[~torch.from_numpy(there)] = -7.0
            assert torch.equal(out.cpu().nan_to_num(11.0), want.nan_to_num(11.0))
        turned = mxfp4.rotate(k.float().cpu().numpy(), at, tab, interleaved)
    for x, cache, scale in zip((turned, v.float().cpu().numpy()), caches, scales):
        codes, s = stored(x, dtype, fmt)
        want = bits_of(torch.full(cache.shape, 9, dtype=kind)) if fmt == "same" else np.full(cache.shape, 9, np.uint8)
        want = want.copy()
        wscale = None if scale is None else np.full(scale.shape, 77, scale.cpu().numpy().dtype)
        for t, slot in enumerate(slots):
            if there[t] and 0 <= slot < pages * page:
                want[slot // page, :, slot % page] = codes[t]
                if scale is not None:
                    wscale[slot // page, :, slot % page] = s[t]
        have = bits_of(cache) if fmt == "same" else cache.cpu().numpy()
        if fmt == "same":     # the payload of a NaN is not specified
            nan = lambda b: np.where(torch.from_numpy(b.view(np.int16).copy()).view(TORCH[dtype]).isnan().numpy(), 0x7FFF, b)
            have, want = nan(have), nan(want)
        if scale is not None:
            assert np.array_equal(np.nan_to_num(scale.cpu().numpy(), nan=-3.0), np.nan_to_num(wscale, nan=-3.0))
        assert np.array_equal(have, want), np.argwhere(have != want)[:5]


FORMATS = pytest.mark.parametrize("fmt", ["same", "e4m3", "mxfp4"])
TYPES = pytest.mark.parametrize("dtype", ["bf16", "f16"])
STYLES = pytest.mark.parametrize("interleaved", [False, True])


@FORMATS
@TYPES
@STYLES
@pytest.mark.parametrize("dim,rotary", [(64, 16), (64, 48), (64, 64), (128, 16), (128, 64), (128, 96), (128, 112), (128, 128)])
def test_rotations(dim, rotary, interleaved, dtype, fmt):
    run_rope(40, 3, 2, dim, rotary, 16, dtype, fmt, interleaved)


@FORMATS
@pytest.mark.parametrize("tokens,hq,hk,dim,page", [(1, 1, 1, 64, 16), (1, 32, 8, 128, 16), (3, 0, 2, 128, 32), (65, 5, 1, 64, 64), (130, 8, 8, 128, 1024), (257, 1, 3, 128, 16)])
def test_sizes(tokens, hq, hk, dim, page, fmt):
    run_rope(tokens, hq, hk, dim, dim, page, "bf16", fmt, False)


@FORMATS
@TYPES
def test_position_zero_is_the_append(dtype, fmt):
    """cos 1 and sin 0: the caches are fp8_kv_append's, bit for bit."""
    tokens, hk, dim, page = 70, 3, 128, 16
    x = normal((tokens, 2 * hk, dim), dtype, 5)
    k, v = x[:, :hk], x[:, hk:]
    slots = torch.randperm(6 * page, device=DEV)[:tokens]
    kind, width = (TORCH[dtype], dim) if fmt == "same" else (torch.uint8, dim if fmt == "e4m3" else dim // 2)
    both = []
    for rope in (False, True):
        caches = [torch.zeros((6, hk, page, width), dtype=kind, device=DEV) for _ in "kv"]
        scales = [None, None] if fmt == "same" else [torch.ones((6, hk, page) + (() if fmt == "e4m3" else (4,)), dtype=torch.float32 if fmt == "e4m3" else torch.uint8, device=DEV) for _ in "kv"]
        if rope:
            fp8.fp8_rope_append(None, k, v, torch.zeros(tokens, dtype=torch.int32, device=DEV), fp8.rope_table(1, dim, device=DEV), slots, *caches, *scales)
        else:
            fp8.fp8_kv_append(k, v, slots, *caches, *scales)
        both.append([t for t in caches + scales if t is not None])
    assert all(torch.equal(a, b) for a, b in zip(*both))


def test_strides():
    """Heads before tokens, and rows that the kernels cannot read in place."""
    tokens, hq, hk, dim = 21, 4, 2, 64
    table, positions = fp8.rope_table(50, dim, device=DEV), i32(np.arange(tokens))
    slots = torch.arange(tokens, device=DEV)
    base = [normal((tokens, h, dim), "bf16", 6 + i) for i, h in enumerate((hq, hk, hk))]
    results = []
    for lay in (lambda t: t, lambda t: t.transpose(0, 1).contiguous().transpose(0, 1), lambda t: torch.cat([t, t[..., :4]], -1)[..., :dim]):
        caches = [torch.zeros((2, hk, 16, dim), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        q, k, v = (lay(t) for t in base)
        results.append([fp8.fp8_rope_append(q, k, v, positions, table, slots, *caches), *caches])
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(results[0], r))


def test_far_positions():
    """A table of 2^20 positions: rows past 2^24 floats; the last position's angles against float64."""
    n, dim = 1 << 20, 128
    table = fp8.rope_table(n, dim, base=500000.0, device=DEV)
    x = normal((2, 1, dim), "bf16", 8)
    positions = i32([n - 1, 123457])
    caches = [torch.zeros((1, 1, 16, dim), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    q = fp8.fp8_rope_append(x, x, x, positions, table, torch.tensor([0, 1], device=DEV), *caches)
    assert torch.equal(q[:, 0], caches[0][0, 0, :2]) and torch.equal(x[:, 0], caches[1][0, 0, :2])
    for t, p in enumerate((n - 1, 123457)):
        angle = p * 500000.0 ** (-2.0 * np.arange(64) / dim)
        z = (f64_of(x)[t, 0, :64] + 1j * f64_of(x)[t, 0, 64:]) * np.exp(1j * angle)
        want = np.concatenate([z.real, z.imag])
        # cosines and sines to 2^-24, two products and a sum in float32, one rounding to bf16
        # a far position's float64 angle is off by 2^-53 of itself: nothing
        bound = 2.0 ** -8 * np.abs(want) + 8 * 2.0 ** -24 * np.tile(np.abs(z), 2)
        assert (np.abs(f64_of(q)[t, 0] - want) <= bound * 1.01).all()


# ------------------------------------------------------------------------- the operators together

def step(s, plan=None, out=None, qout=None):
    plan = fp8.fp8_paged_plan(s["cached"], s["added"], s["table"], s["free"], s["taken"], s["t"], s["page"], out=plan)
    q = fp8.fp8_rope_append(s["q"], s["k"], s["v"], plan.positions, s["turn"], plan.slots, *s["caches"], out=qout)
    return plan, q, fp8.fp8_attn_paged(q, *s["caches"][:2], s["table"], plan.seq_lens, plan.cu_tokens, *s["caches"][2:], max_new=40, out=out)


@pytest.mark.parametrize("fmt", ["same", "e4m3", "mxfp4"])
def test_step_eager_on_another_stream_and_in_a_graph(fmt):
    """Plan, rotation with append and attention of two steps over one cache: the second one eager, on a side stream and in a
    graph that is replayed with eager work between, with padded token buffers; and against float64."""
    hq, hk, dim, page, dtype = 8, 2, 128, 16, "bf16"
    first, added = [70, 5, 0, 33], [1, 1, 40, 1]
    pages = 20
    kind, width = (TORCH[dtype], dim) if fmt == "same" else (torch.uint8, dim if fmt == "e4m3" else dim // 2)
    caches = [torch.zeros((pages, hk, page, width), dtype=kind, device=DEV) for _ in "kv"]
    if fmt != "same":
        caches += [torch.zeros((pages, hk, page) + (() if fmt == "e4m3" else (4,)), dtype=torch.float32 if fmt == "e4m3" else torch.uint8, device=DEV) for _ in "kv"]
    else:
        caches += [None, None]
    s = dict(page=page, caches=caches, turn=fp8.rope_table(128, dim, device=DEV), free=torch.randperm(pages, device=DEV).int(),
             table=torch.full((4, 8), -1, dtype=torch.int32, device=DEV))
    x0 = normal((sum(first), hq + 2 * hk, dim), dtype, 30)
    s.update(cached=i32([0] * 4), added=i32(first), taken=i32([0]), t=sum(first), q=x0[:, :hq], k=x0[:, hq:hq + hk], v=x0[:, hq + hk:])
    plan, _, _ = step(s)
    pad = 5                                                           # a fixed token count, more than there are tokens
    x = normal((sum(added) + pad, hq + 2 * hk, dim), dtype, 31)
    s.update(cached=plan.seq_lens, added=i32(added), taken=plan.taken, t=sum(added) + pad, q=x[:, :hq], k=x[:, hq:hq + hk], v=x[:, hq + hk:])
    before = s["table"].clone()
    plan, q, want = step(s)
    torch.cuda.synchronize()
    n = sum(added)
    keep = [y.clone() for y in (*plan, s["table"], q[:n], want[:n], *[c for c in caches if c is not None])]

    def check(plan, q, out, what):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*plan, s["table"], q[:n], out[:n], *[c for c in caches if c is not None]), keep)), what

    side = torch.cuda.Stream()
    s["table"].copy_(before)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(s)
    check(*got, "side stream")
    bufs, out, qout = fp8.paged_plan_buffers(4, s["t"], DEV), torch.empty_like(want), torch.empty_like(want)
    s["table"].copy_(before)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s, bufs, out, qout)
    for rep in range(4):
        out.fill_(7.0)
        qout.fill_(5.0)
        s["table"].copy_(before)
        torch.cuda.synchronize()
        graph.replay()
        check(bufs, qout, out, rep)
        assert (out[n:] == 7.0).all() and (qout[n:] == 5.0).all()     # rows behind the last sequence
        _ = (want.float() * 2).sum()
    # against float64: what the cache holds, with the rotated queries
    cache = Cache4([c + a for c, a in zip(first, added)], hk, dim, page, 1)
    cache.table = s["table"].cpu().numpy()
    for i, name in enumerate("kv"):
        c = caches[i]
        if fmt == "same":
            cache.values[name] = f64_of(c)
        elif fmt == "e4m3":
            cache.values[name] = decode_e4m3(c.cpu().numpy()).astype(np.float64) * f64_of(caches[2 + i])[..., None]
        else:
            cache.values[name] = mxfp4.decode(c.cpu().numpy(), caches[2 + i].cpu().numpy())
    check_paged(q[:n], cache, added, want[:n], None, dtype, 1 / math.sqrt(dim), 0)
    if fmt == "same":     # and the cache against the definition: the second step's keys of request 2, at positions 0 .. 39
        angle = np.arange(40)[:, None] * 10000.0 ** (-2.0 * np.arange(64) / dim)
        kk = f64_of(s["k"][2:42])
        z = (kk[..., :64] + 1j * kk[..., 64:]) * np.exp(1j * angle)[:, None]
        full = np.concatenate([z.real, z.imag], -1)
        mag = np.tile(np.abs(z), 2)
        assert (np.abs(cache.request("k", 2) - full) <= 2.0 ** -8 * 1.01 * np.abs(full) + 8 * 2.0 ** -24 * mag).all()
