"""Attention over a paged cache in four bits, and the appends into it, against float64 references: at
the sizes, masks and scales where they can go wrong.  With bf16 every stored value is a number of the
type, so the bounds are those of a 16-bit cache (oracle.serving.attention_bound)."""

import math

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from mxfp4_util import Cache4
from oracle import mxfp4
from oracle.serving import attention_ref
from parity_util import DEV
from serving_util import TORCH, check_paged, check_rows, cu_of, f64_of, normal

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 64, 16), (1, 8, 128, 16), (33, 3, 64, 32), (130, 8, 128, 64), (515, 2, 128, 1024)])
def test_append(dtype, tokens, heads, dim, page):
    rng = np.random.default_rng(tokens)
    fused = normal((tokens, 3 * heads + 1, dim), dtype, tokens, 3.0)
    k, v = fused[:, 1:1 + heads], fused[:, 1 + 2 * heads:]
    if tokens > 8:
        k[1] = 0.0                                                       # scale 1
        k[2, 0, 5], v[3, 0, 0], v[3, 0, 40] = float("nan"), float("inf"), float("-inf")
        v[4] *= 2.0 ** -18                                               # subnormal fp16
        k[5] = torch.finfo(TORCH[dtype]).max                             # codes of 3 rather than infinity
        k[6, :, ::2] = torch.finfo(TORCH[dtype]).max * 0.8
        v[6] = torch.finfo(TORCH[dtype]).tiny
        v[7] = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25], dtype=v.dtype, device=DEV).repeat(dim // 8)   # ties
    pages = -(-tokens // page) + 2
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 8:
        slots[-1], slots[-2], slots[0] = -1, pages * page, -(1 << 40)    # skipped
    caches = [torch.full((pages, heads, page, dim // 2), 9, dtype=torch.uint8, device=DEV) for _ in "kv"]
    scales = [torch.full((pages, heads, page, dim // 32), 77, dtype=torch.uint8, device=DEV) for _ in "kv"]
    fp8.fp8_kv_append(k, v, torch.from_numpy(slots).to(DEV), *caches, *scales)
    torch.cuda.synchronize()
    for x, cache, scale in zip((k, v), caches, scales):
        want, wscale = np.full(cache.shape, 9, np.uint8), np.full(scale.shape, 77, np.uint8)
        codes, s = mxfp4.quantize(f64_of(x), dtype)
        for t, slot in enumerate(slots):
            if 0 <= slot < pages * page:
                want[slot // page, :, slot % page], wscale[slot // page, :, slot % page] = codes[t], s[t]
        assert np.array_equal(scale.cpu().numpy(), wscale)
        assert np.array_equal(cache.cpu().numpy(), want)


# ------------------------------------------------------------------------------------- attention

def run4(lens, new, hq, hk, dim, page, dtype, window=0, seed=0, max_new=None, width=None):
    cache = Cache4(lens, hk, dim, page, seed + 1, width=width)
    t = sum(new)
    q = normal((t, hq + 1, dim), dtype, seed)[:, 1:]
    full = torch.full((t * hq * dim + 512,), -7.0, dtype=TORCH[dtype], device=DEV)
    out = full[: t * hq * dim].view(t, hq, dim)
    kw = dict(window=window, max_new=max(new) if max_new is None else max_new)
    args = (q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of(new), cache.ks, cache.vs)
    _, lse = fp8.fp8_attn_paged(*args, out=out, return_lse=True, **kw)
    torch.cuda.synchronize()
    assert (full[t * hq * dim:] == -7.0).all()
    check_paged(q, cache, new, out, lse, dtype, 1 / math.sqrt(dim), window)
    assert torch.equal(fp8.fp8_attn_paged(*args, **kw), out)
    return cache, q, out


TYPES = pytest.mark.parametrize("dtype", ["bf16", "f16"])
DIMS = pytest.mark.parametrize("dim", [64, 128])


@TYPES
@DIMS
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_single_tokens(page, dim, dtype):
    run4([1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1025], [1] * 18, 8, 2, dim, page, dtype)


@TYPES
@DIMS
@pytest.mark.parametrize("page", [16, 32, 128])
def test_chunks(page, dim, dtype):
    run4([1, 40, 64, 129, 200, 333], [1, 40, 2, 100, 33, 70], 4, 2, dim, page, dtype)      # many rows
    run4([9, 40, 64, 129, 200, 333], [9, 10, 2, 7, 13, 8], 8, 2, dim, page, dtype)         # few, two tokens' rows and more a tile
    run4([9, 40, 64, 129, 200, 333], [3, 2, 2, 7, 1, 8], 4, 2, dim, page, dtype)           # few


@pytest.mark.parametrize("hq,hk", [(1, 1), (5, 1), (8, 1), (16, 2), (32, 32), (40, 1), (64, 1), (12, 4)])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 7, 3]])
def test_heads(hq, hk, new):
    run4([9, 100, 257], new, hq, hk, 128, 16, "bf16", seed=hq)


@pytest.mark.parametrize("window", [1, 15, 16, 40, 128, 1000])
@TYPES
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 9, 14], [1, 60, 90]])
def test_windows(window, dtype, new):
    run4([5, 260, 700], new, 8, 2, 128, 32, dtype, window=window)


@TYPES
def test_long(dtype):
    """Few rows over a long axis: the work is split and joined."""
    run4([9000, 3, 2500], [1, 1, 1], 8, 2, 128, 64, dtype)
    run4([5000], [2], 2, 2, 64, 16, dtype)
    run4([9000, 3, 2500], [5, 3, 6], 8, 2, 128, 64, dtype)
    run4([4000], [150], 4, 1, 128, 16, dtype)


@pytest.mark.parametrize("dim,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("requests,kv_heads,window", [(24, 64, 0), (90, 32, 0), (90, 16, 500), (3, 256, 0)])
def test_many_steps(requests, kv_heads, window, dim, dtype):
    """Several pieces of 256 keys a workgroup, cut wherever they end: few workgroups a key head."""
    rng = np.random.default_rng(requests)
    lens = [int(x) for x in rng.choice([1, 5, 255, 256, 257, 511, 700, 1300, 2100], requests)]
    lens[-1] = 1800
    run4(lens, [0 if r % 11 == 3 else 1 for r in range(requests)], kv_heads, kv_heads, dim, 16, dtype, window=window)


@TYPES
@pytest.mark.parametrize("dim,window", [(64, 0), (128, 0), (64, 300)])
@pytest.mark.parametrize("many", [False, True])
def test_mixed(many, dim, window, dtype):
    lens = [3000, 1, 900, 40, 128, 2000, 17, 1, 64, 333, 1500, 256] * (7 if many else 1)
    new = [100, 1, 1, 1, 1, 3, 1, 1, 0, 1, 17, 1] * (7 if many else 1)
    run4(lens, new, 8, 2, dim, 16, dtype, window=window)
    new = [4, 1, 1, 1, 1, 3, 1, 1, 0, 1, 5, 1] * (7 if many else 1)
    run4(lens, new, 8, 2, dim, 16, dtype, window=window)


@pytest.mark.parametrize("max_new", [0, 1, 64, 4096])
def test_hint_changes_no_meaning(max_new):
    run4([100, 300, 64], [1, 130, 0], 8, 2, 128, 16, "bf16", max_new=max_new)


def test_wide_table_and_many_requests():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 200, 300)]
    run4(lens, [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 3, 300))], 4, 1, 64, 16, "f16", width=100)
    run4(lens * 4, [1] * 1200, 4, 1, 64, 16, "bf16")       # more than are cut


@DIMS
@pytest.mark.parametrize("new", [[3, 2, 4], [8, 3, 9], [40, 70, 90]])
def test_rows_without_keys(dim, new):
    lens = [1, 0, 66]
    cache = Cache4(lens, 2, dim, 16, 5)
    q = normal((sum(new), 4, dim), "bf16", 6)
    out, lse = fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of(new), cache.ks, cache.vs, max_new=max(new), return_lse=True)
    check_paged(q, cache, new, out, lse, "bf16", 1 / math.sqrt(dim), 0, rel=False)
    assert (out[new[0]:new[0] + new[1]] == 0).all() and lse[new[0]:new[0] + new[1]].isneginf().all()


@pytest.mark.parametrize("new", [1, 10, 60])
def test_pages_that_do_not_exist(new):
    """Table entries outside the cache read as zero keys and values."""
    cache = Cache4([80, 70], 2, 128, 16, 9)
    q = normal((2 * new, 4, 128), "bf16", 10)
    table = cache.dev_table.clone()
    table[0, 2], table[1, 0], table[1, 4] = -1, 1 << 30, cache.k.shape[0]
    out = fp8.fp8_attn_paged(q, cache.k, cache.v, table, cache.dev_lens, cu_of([new, new]), cache.ks, cache.vs, max_new=new)
    for r, holes in enumerate(([(32, 48)], [(0, 16), (64, 70)])):
        kk, vv = cache.request("k", r).copy(), cache.request("v", r).copy()
        for lo, hi in holes:
            kk[lo:hi], vv[lo:hi] = 0, 0
        s = slice(r * new, (r + 1) * new)
        check_rows(out[s], None, attention_ref(f64_of(q[s]), kk, vv, len(kk) - new, 1 / math.sqrt(128), 0), "bf16", len(kk), 128, 6.0, f"request {r}")


def test_lengths_beyond_their_tensors_stay_inside():
    cache = Cache4([64], 2, 64, 16, 11, width=4)
    q = normal((10, 2, 64), "bf16", 12)
    out = torch.full((10, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, i32([1 << 30]), i32([-4, 6]), cache.ks, cache.vs, out=out, max_new=6)
    check_paged(q[:6], cache, [6], out[:6], None, "bf16", 1 / 8, 0)
    assert (out[6:] == 3.0).all()


@TYPES
@pytest.mark.parametrize("group", [1, 20, 70])
def test_every_code_at_every_scale(group, dtype):
    """Requests of one key and queries of zeros, so that its weight is exactly 1: the output is the value as a number of
    the type, for all codes at all 256 scale bytes; past the type's range infinite, with byte 255 NaN."""
    n, dim, page = 256, 64, 16
    cache = Cache4([1] * n, 1, dim, page, 19)
    i = torch.arange(32)                                           # every code in both halves of a byte
    codes = (i % 16 | (i * 7 + i // 16 * 3) % 16 << 4).to(torch.uint8).to(DEV)
    for r in range(n):
        at = int(cache.table[r, 0])
        cache.v[at, 0, 0], cache.vs[at, 0, 0] = codes, r
    q = normal((n, group, dim), dtype, 20, 0.0)
    out = fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of([1] * n), cache.ks, cache.vs, max_new=1)
    exact = mxfp4.decode(np.repeat(codes.cpu().numpy()[None], n, 0), np.repeat(np.arange(n, dtype=np.uint8)[:, None], 2, 1))
    want = torch.from_numpy(exact).to(TORCH[dtype]).double()
    got = out.double().cpu()
    assert (got[255].isnan()).all()
    hit = want[:, None].expand_as(got)
    # float32 sums of the matrix unit may flush what lies below 2^-126 to zero
    ok = (got == hit) | ((hit.abs() < 2.0 ** -126) & (got == 0)) | (hit.isnan() & got.isnan())
    assert ok[:255].all(), (~ok[:255]).nonzero()[:5]


@TYPES
@pytest.mark.parametrize("new", [1, 10, 60])
def test_scales_far_apart(new, dtype):
    """Blocks whose scales differ by up to 2^12 inside a key and between keys."""
    cache = Cache4([300, 900], 2, 128, 16, 23, low=116, high=128)
    cache.ks[:] = cache.ks.clamp(max=125)
    cache.reread()
    q = normal((2 * new, 8, 128), dtype, 24)
    out, lse = fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of([new] * 2), cache.ks, cache.vs, max_new=new, return_lse=True)
    check_paged(q, cache, [new] * 2, out, lse, dtype, 1 / math.sqrt(128), 0)


# ---------------------------------------------------------------------- values that are not finite

def same(a, b):
    kind = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def attend(cache, q, new, window=0):
    out, lse = fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of(new), cache.ks, cache.vs, max_new=max(new),
                                  window=window, return_lse=True)
    torch.cuda.synchronize()
    return out, lse


@TYPES
@DIMS
@pytest.mark.parametrize("new", [3, 14, 90])
@pytest.mark.parametrize("length", [130, 3000])
def test_blocks_of_nan(length, new, dim, dtype):
    """A late token's block is NaN: rows before it and the other key head keep their bits; of the rows that see it, a value
    spoils its 32 channels and nothing else, a key everything."""
    q = normal((new, 8, dim), dtype, 22)
    for name in "vk":
        cache = Cache4([length], 2, dim, 16, 21)
        good, good_lse = attend(cache, q, [new])
        page, at = cache.place(0, length - 2)
        getattr(cache, name + "s")[page, 1, at, 1] = 255
        out, lse = attend(cache, q, [new])
        assert same(out[:-2], good[:-2]) and same(out[:, :4], good[:, :4])
        assert same(lse[:-2], good_lse[:-2]) and same(lse[:, :4], good_lse[:, :4])
        if name == "v":
            assert same(lse, good_lse) and out[-2:, 4:, 32:64].isnan().all()
            assert same(out[-2:, 4:, :32], good[-2:, 4:, :32]) and same(out[-2:, 4:, 64:], good[-2:, 4:, 64:])
        else:
            assert out[-2:, 4:].isnan().all() and lse[-2:, 4:].isnan().all()


@DIMS
@pytest.mark.parametrize("new", [3, 14, 90])
@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("byte", [255, 250])
def test_before_the_window_nothing_matters(byte, name, new, dim):
    window, length = 40, 230
    q = normal((new, 8, dim), "f16", 26)
    cache = Cache4([length], 2, dim, 16, 25)
    good, good_lse = attend(cache, q, [new], window)
    page, at = cache.place(0, length - new - window)
    getattr(cache, name + "s")[page, :, at] = byte                # NaN, and infinite in fp16
    out, lse = attend(cache, q, [new], window)
    assert same(out, good) and same(lse, good_lse)


@pytest.mark.parametrize("new", [3, 14, 90])
def test_values_past_fp16(new):
    """Infinite in fp16: positive and negative channels by their sign, for the rows that see them."""
    q = normal((new, 4, 64), "f16", 28)
    cache = Cache4([150], 1, 64, 16, 27)
    good, _ = attend(cache, q, [new])
    page, at = cache.place(0, 149)
    cache.v[page, 0, at], cache.vs[page, 0, at] = 0x9A, 150       # channels 2 i: -1, 2 i + 1: -0.5 ... times 2^23
    out, _ = attend(cache, q, [new])
    assert same(out[:-1], good[:-1]) and out[-1].isneginf().all()
    cache.v[page, 0, at, 3] = 0x27                                 # channel 6: 6, channel 7: 1
    out, _ = attend(cache, q, [new])
    assert (out[-1, :, 6:8] == math.inf).all() and out[-1, :, 8:].isneginf().all()


# ------------------------------------------------------------------- offsets, streams, workspaces

def test_cache_beyond_32_bit_offsets():
    """Pages whose code bytes lie past 4 GiB of the cache: appended to and read by each kernel."""
    hk, dim, page = 8, 128, 1024
    pages = (1 << 32) // (hk * page * dim // 2) + 40
    kc, vc = (torch.empty((pages, hk, page, dim // 2), dtype=torch.uint8, device=DEV) for _ in "kv")
    ks, vs = (torch.empty((pages, hk, page, dim // 32), dtype=torch.uint8, device=DEV) for _ in "kv")
    n = 1500
    x = normal((n, 2 * hk, dim), "bf16", 41)
    k, v = x[:, :hk], x[:, hk:]
    table = i32([[pages - 1, pages - 37]])
    t = torch.arange(n, device=DEV)
    slots = table[0, t // page].long() * page + t % page
    turn = fp8.rope_table(2, 128, device=DEV)
    fp8.fp8_rope_append(None, k, v, torch.zeros(n, dtype=torch.int32, device=DEV), turn, slots, kc, vc, ks, vs)     # position 0: as they are
    kk, vv = (mxfp4.decode(*mxfp4.quantize(f64_of(y), "bf16")) for y in (k, v))
    for new in (1, 8, 30):
        q = normal((new, 16, dim), "bf16", 42 + new)
        out = fp8.fp8_attn_paged(q, kc, vc, table, i32([n]), i32([0, new]), ks, vs, max_new=new)
        check_rows(out, None, attention_ref(f64_of(q), kk, vv, n - new, 1 / math.sqrt(dim), 0), "bf16", n, dim, float(np.abs(vv).max()), f"{new} new")


@pytest.mark.parametrize("new", [[1, 1, 1], [5, 9, 4], [1, 50, 90]])
def test_workspace_serves_every_format(new):
    """One workspace for calls over 4 bits and 16 bits in turn; decreasing cu_tokens leave it fit."""
    from serving_util import Cache
    lens = [600, 3000, 900]
    c4, c16 = Cache4(lens, 2, 128, 16, 51), Cache(lens, 2, 128, 16, "bf16", False, 52)
    q = normal((sum(new), 8, 128), "bf16", 53)
    need = fp8.fp8_attn_paged_workspace(sum(new), 3, 8, 2, 128, c4.dev_table.shape[1], 16, max(new))
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device=DEV)
    ws[:16384] = 0
    args4 = (q, c4.k, c4.v, c4.dev_table, c4.dev_lens)
    args16 = (q, c16.k, c16.v, c16.dev_table, c16.dev_lens)
    kw = dict(max_new=max(new), workspace=ws)
    want4 = fp8.fp8_attn_paged(*args4, cu_of(new), c4.ks, c4.vs, max_new=max(new))
    want16 = fp8.fp8_attn_paged(*args16, cu_of(new), max_new=max(new))
    for cu in ([0, sum(new), 0, sum(new)], [5, -3, 1 << 30, 7]):
        fp8.fp8_attn_paged(*args4, i32(cu), c4.ks, c4.vs, **kw)
        assert torch.equal(fp8.fp8_attn_paged(*args16, cu_of(new), **kw), want16)
        assert torch.equal(fp8.fp8_attn_paged(*args4, cu_of(new), c4.ks, c4.vs, **kw), want4)
    assert not ws[:16384].any()
    with pytest.raises(fp8.Fp8Error, match="BAD_SHAPE"):
        fp8.fp8_attn_paged(*args4, cu_of(new), c4.ks, c4.vs, max_new=max(new), workspace=ws[: need - 1])


def test_each_request_is_what_it_is_alone():
    """Requests that share workgroups keep their bits."""
    batch = 700
    lens = [180 if r % 2 else 200 for r in range(batch)]
    cache = Cache4(lens, 2, 64, 16, 5, width=20)
    for r in range(0, batch, 2):
        page, at = cache.place(r, lens[r] - 1)
        cache.vs[page, :, at] = (255, 140)[r // 2 % 2]
    q = normal((batch, 8, 64), "bf16", 6)
    out = fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of([1] * batch), cache.ks, cache.vs, max_new=1)
    for r in (0, 1, 2, 3, 301, 303, 699):
        alone = fp8.fp8_attn_paged(q[r:r + 1], cache.k, cache.v, cache.dev_table[r:r + 1, :13].contiguous(), cache.dev_lens[r:r + 1], cu_of([1]),
                                   cache.ks, cache.vs, max_new=1)
        assert same(out[r:r + 1], alone), r
    assert out[1::2].isfinite().all()


def test_two_streams_at_once():
    cache = Cache4([6000, 100], 4, 128, 16, 81)
    qs = [normal((2, 16, 128), "bf16", 82 + i) for i in range(2)]
    args = (cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of([1, 1]), cache.ks, cache.vs)
    want = [fp8.fp8_attn_paged(q, *args, max_new=1) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fp8.fp8_attn_paged(qs[i], *args, max_new=1))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for os_, w in zip(got, want) for o in os_)


def test_types_of_torch_for_codes_and_scales():
    """float4_e2m1fn_x2 and float8_e8m0fnu tensors are what uint8 ones are."""
    cache = Cache4([100], 2, 64, 16, 91)
    q = normal((1, 4, 64), "bf16", 92)
    want = fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of([1]), cache.ks, cache.vs)
    got = fp8.fp8_attn_paged(q, cache.k.view(torch.float4_e2m1fn_x2), cache.v.view(torch.float4_e2m1fn_x2), cache.dev_table, cache.dev_lens,
                             cu_of([1]), cache.ks.view(torch.float8_e8m0fnu), cache.vs.view(torch.float8_e8m0fnu))
    assert torch.equal(got, want)
