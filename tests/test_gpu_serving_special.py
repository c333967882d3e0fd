"""Attention over a paged cache where requests and rows must not reach each other: pages that do not
exist next to scales that are not finite, value scales far apart, and keys and values that are not
finite in places that some rows see and others do not.  Float64 references as in test_gpu_serving.py."""

import math

import numpy as np
import pytest
import torch

import fp8_quantized_gemm_amax_amd as fp8
from oracle import decode_e4m3
from oracle.serving import attention_ref
from parity_util import DEV
from serving_util import Cache, check_rows, cu_of, f64_of, normal

pytestmark = pytest.mark.gpu


def set_row(cache, name, r, token, codes=None, scale=None):
    """Overwrites a token of request r in an e4m3 cache (every head): its codes, its scale."""
    page, at = int(cache.table[r, token // cache.page]), token % cache.page
    if codes is not None:
        getattr(cache, name)[page, :, at] = codes
    if scale is not None:
        getattr(cache, name + "s")[page, :, at] = scale


def reread(cache):
    """The cache's values from what its tensors hold now."""
    for n in "kv":
        c, s = (x.cpu().numpy() for x in (getattr(cache, n), getattr(cache, n + "s")))
        cache.values[n] = decode_e4m3(c).astype(np.float64) * s.astype(np.float64)[..., None]


# ------------------------------------------------- several requests of one workgroup, e4m3 scales

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_missing_pages_next_to_scales_that_are_not_finite(dim, dtype):
    """More requests than workgroups, so that a workgroup takes several: every second request has a key and
    a value whose scale is NaN or infinite, the others lack the page at the same place, which reads as zero."""
    batch, n, page, hk = 700, 70, 16, 2
    cache = Cache([n] * batch, hk, dim, page, dtype, True, 3, width=20)
    table = cache.dev_table.clone()
    odd = list(range(1, batch, 2))
    for r in range(0, batch, 2):
        bad = (float("nan"), float("inf"))[r // 2 % 2]
        for token in (20, 66):
            set_row(cache, "kv"[r // 4 % 2], r, token, scale=bad)
    table[odd, 1] = -1
    table[odd, 4] = 1 << 30
    q = normal((batch, 4 * hk, dim), dtype, 4)
    out = fp8.fp8_attn_paged(q, cache.k, cache.v, table, cache.dev_lens, cu_of([1] * batch), cache.ks, cache.vs, max_new=1)
    assert out[odd].isfinite().all()
    for r in odd[:60:7] + odd[-40::7]:
        kk, vv = cache.request("k", r).copy(), cache.request("v", r).copy()
        for x in (kk, vv):
            x[16:32], x[64:70] = 0, 0
        ref = attention_ref(f64_of(q[r:r + 1]), kk, vv, n - 1, 1 / math.sqrt(dim), 0)
        check_rows(out[r:r + 1], None, ref, dtype, n, dim, float(np.abs(vv).max()), f"request {r}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_requests_whose_value_scales_lie_far_apart(dim, dtype):
    """Neighbours in a workgroup with value scales 2^14 apart: each is as exact as it is alone, bit for bit."""
    batch, page, hk = 700, 16, 2
    lens = [180 if r % 2 else 200 for r in range(batch)]
    cache = Cache(lens, hk, dim, page, dtype, True, 5, width=20)
    for r in range(0, batch, 2):
        pages = torch.from_numpy(cache.table[r, : -(-lens[r] // page)].astype(np.int64)).to(DEV)
        cache.vs[pages] *= 2.0 ** 14
    reread(cache)
    q = normal((batch, 4 * hk, dim), dtype, 6)
    args = (cache.k, cache.v)
    out = fp8.fp8_attn_paged(q, *args, cache.dev_table, cache.dev_lens, cu_of([1] * batch), cache.ks, cache.vs, max_new=1)
    for r in (1, 2, 3, 301, 303, 699):
        kk, vv = cache.request("k", r), cache.request("v", r)
        ref = attention_ref(f64_of(q[r:r + 1]), kk, vv, lens[r] - 1, 1 / math.sqrt(dim), 0)
        check_rows(out[r:r + 1], None, ref, dtype, lens[r], dim, 0.0, f"request {r}")
        alone = fp8.fp8_attn_paged(q[r:r + 1], *args, cache.dev_table[r:r + 1, :13].contiguous(), cache.dev_lens[r:r + 1], cu_of([1]),
                                   cache.ks, cache.vs, max_new=1)
        assert torch.equal(out[r:r + 1], alone), r


# ------------------------------------------------------------- fp16 queries over e4m3 value scales

def few_or_many(many):
    """New tokens of one request: rows that go to the kernel for few (4 a token and key head) and for many."""
    return 90 if many else 6


def paged(cache, q, new, **kw):
    return fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of(new), cache.ks, cache.vs, max_new=max(new), **kw)


def check_request(cache, q, out, dim, window=0, dtype="f16"):
    """One request's rows, each against the values it sees.  The weights carry 16 bits in float32's range, so nothing in
    the bound goes by the largest value (vmax 0)."""
    kk, vv = cache.request("k", 0), cache.request("v", 0)
    ref = attention_ref(f64_of(q), kk, vv, len(kk) - len(q), 1 / math.sqrt(dim), window)
    check_rows(out, None, ref, dtype, len(kk), dim, 0.0, "request", rel=False)
    for i in range(len(q)):      # row by row as well, since their sizes may differ; 2^-25: half the spacing of fp16's smallest
        w = ref[0][i]
        assert np.linalg.norm(f64_of(out[i]) - w) <= 2 * 2.0 ** -11 * np.linalg.norm(w) + math.sqrt(w.size) * 2.0 ** -25, i


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("length", [130, 1500])
def test_a_late_value_of_large_scale_reaches_only_its_rows(length, many, dim):
    """The last new token's value scale is 2^18 times the others': the rows before it keep their bits and their exactness."""
    new = few_or_many(many)
    cache = Cache([length], 2, dim, 16, "f16", True, 11)
    cache.vs *= 2.0 ** -10
    q = normal((new, 8, dim), "f16", 12)
    before = paged(cache, q, [new])
    set_row(cache, "v", 0, length - 1, scale=cache.vs[int(cache.table[0, (length - 1) // 16]), :, (length - 1) % 16] * 2.0 ** 18)
    reread(cache)
    out = paged(cache, q, [new])
    assert torch.equal(out[:-1], before[:-1])
    check_request(cache, q, out, dim)


@pytest.mark.parametrize("scale", [2.0 ** 24, float("inf"), float("nan")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("many", [False, True])
def test_a_value_before_the_window_does_not_matter(many, dim, scale):
    """A key that no row's window reaches, in a tile that some of their keys share."""
    new, window = few_or_many(many), 40
    cache = Cache([230], 2, dim, 16, "f16", True, 13)
    cache.vs *= 2.0 ** -14
    reread(cache)
    q = normal((new, 8, dim), "f16", 14)
    before = paged(cache, q, [new], window=window)
    set_row(cache, "v", 0, 230 - new - window, scale=scale)
    assert torch.equal(paged(cache, q, [new], window=window), before)
    check_request(cache, q, before, dim, window)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("zero", [False, True])
def test_a_seen_value_of_large_scale_and_no_weight(zero, many, dim):
    """Seen by every row: a value row of zeros, whose scale is 1, among values of scale 2^-14; or a value whose scale is
    2^20 times the others' under a key whose weight all but vanishes."""
    new = few_or_many(many)
    cache = Cache([150], 2, dim, 16, "f16", True, 15)
    cache.vs *= 2.0 ** -14
    q = normal((new, 8, dim), "f16", 16, 0.1)
    if zero:
        set_row(cache, "v", 0, 7, codes=0, scale=1.0)
    else:   # a key against the queries' common part: score about -25
        q = q + torch.ones(dim, dtype=q.dtype, device=DEV)
        set_row(cache, "k", 0, 7, codes=0xB8, scale=25.0 / math.sqrt(dim))      # 0xB8: -1
        set_row(cache, "v", 0, 7, scale=2.0 ** 6)
    reread(cache)
    check_request(cache, q, paged(cache, q, [new]), dim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("length", [130, 1500])
def test_value_scales_beyond_fp16(length, many, dim):
    """Scales up to 2^24 whose codes are small enough for fp16 outputs (a cache that bf16 rows were appended to): at two
    places that every row sees, and at the last token, which reaches only its own row."""
    new = few_or_many(many)
    cache = Cache([length], 2, dim, 16, "f16", True, 17)
    q = normal((new, 8, dim), "f16", 18)
    small = torch.arange(dim, device=DEV).remainder(8).to(torch.uint8) | torch.arange(dim, device=DEV).remainder(3).eq(0).to(torch.uint8) * 0x80
    set_row(cache, "v", 0, 7, codes=small, scale=2.0 ** 21)          # codes of up to 7 / 512
    set_row(cache, "v", 0, 33, codes=small.flip(0), scale=2.0 ** 22)
    before = paged(cache, q, [new])
    set_row(cache, "v", 0, length - 1, codes=small, scale=2.0 ** 24)
    reread(cache)
    out = paged(cache, q, [new])
    assert torch.equal(out[:-1], before[:-1])
    check_request(cache, q, out, dim)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [1, 70])
def test_every_code_at_every_power_of_two(group, dtype):
    """Requests of one key and queries of zeros, so that its weight is exactly 1: the output is the value, code times scale,
    rounded once, for every finite code and the scales 2^-24 .. 2^7.  70 rows a request go to the kernel for many rows."""
    n, dim, page = 32, 128, 16
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F] + [0, 0x80], dtype=torch.uint8, device=DEV).view(2, dim)
    cache = Cache([1] * n, 2, dim, page, dtype, True, 19)
    for r in range(n):
        at = int(cache.table[r, 0])
        cache.v[at, :, 0], cache.vs[at, :, 0] = codes, 2.0 ** (r - 24)
    q = normal((n, 2 * group, dim), dtype, 20, 0.0)
    out = fp8.fp8_attn_paged(q, cache.k, cache.v, cache.dev_table, cache.dev_lens, cu_of([1] * n), cache.ks, cache.vs, max_new=1)
    exact = decode_e4m3(codes.cpu().numpy()).astype(np.float64)[None] * 2.0 ** (np.arange(n)[:, None, None] - 24)
    want = torch.from_numpy(exact).to(q.dtype).repeat_interleave(group, dim=1).to(DEV)
    assert torch.equal(out, want)


# ------------------------------------------------- keys and values that are not finite, paged caches

BAD = {"nan": float("nan"), "inf": float("inf"), "-inf": float("-inf")}
KINDS = [("bf16", False), ("bf16", True), ("f16", False), ("f16", True)]


def run_bits(cache, q, new, window=0):
    out, lse = paged(cache, q, [new], window=window, return_lse=True)
    torch.cuda.synchronize()
    return out, lse


def same(a, b):
    """The same bits, NaN among them."""
    return torch.equal(a.contiguous().view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.contiguous().view(torch.int16 if b.element_size() == 2 else torch.int32))


def spoil(cache, name, token, head, channel, what):
    """Puts a value that is not finite into one head's row of a token: in a 16-bit cache one channel; in an e4m3 one the
    code of NaN in one channel ("code"), or the row's scale."""
    page, at = int(cache.table[0, token // cache.page]), token % cache.page
    if not cache.e4m3:
        getattr(cache, name)[page, head, at, channel] = BAD[what]
    elif what == "code":
        getattr(cache, name)[page, head, at, channel] = 0xFF
    else:
        getattr(cache, name + "s")[page, head, at] = BAD[what]


@pytest.mark.parametrize("dtype,e4m3", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("length", [130, 3000])
def test_values_that_are_not_finite(length, many, dim, dtype, e4m3):
    """A late token's value: the rows before it and the other key head keep their bits, the rows that see it get the IEEE
    result.  130 keys are walked whole, 3000 are cut into pieces that are joined."""
    new = few_or_many(many)
    q = normal((new, 8, dim), dtype, 22)
    for what in ("nan", "inf", "-inf") if not e4m3 else ("nan", "inf", "code"):
        cache = Cache([length], 2, dim, 16, dtype, e4m3, 21)
        good, good_lse = run_bits(cache, q, new)
        at = length - 3
        spoil(cache, "v", at, 1, 7, what)
        out, lse = run_bits(cache, q, new)
        assert same(lse, good_lse), what
        assert same(out[:-3], good[:-3]) and same(out[:, :4], good[:, :4]), what
        hit = out[-3:, 4:]
        if e4m3 and what != "code":
            codes = cache.v[int(cache.table[0, at // 16]), 1, at % 16].cpu()
            want = torch.from_numpy(decode_e4m3(codes.numpy())).float() * BAD[what]
            assert torch.equal(hit.float().cpu().nan_to_num(7.0, 8.0, -8.0), want.nan_to_num(7.0, 8.0, -8.0).expand(hit.shape)), what
        else:
            want = torch.full_like(hit[..., 7].float(), BAD["nan" if what == "code" else what])
            assert torch.equal(hit[..., 7].float().nan_to_num(7.0, 8.0, -8.0), want.nan_to_num(7.0, 8.0, -8.0)), what
            rest = [c for c in range(dim) if c != 7]
            assert same(hit[..., rest], good[-3:, 4:][..., rest]), what


@pytest.mark.parametrize("dtype,e4m3", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("length", [130, 3000])
def test_keys_that_are_not_finite(length, many, dim, dtype, e4m3):
    """A late token's key: a score of NaN or +inf gives NaN, one of -inf no weight; rows that do not see it keep their bits."""
    new = few_or_many(many)
    q = normal((new, 8, dim), dtype, 24)
    for what in ("nan", "inf", "-inf") if not e4m3 else ("nan", "inf", "code"):
        cache = Cache([length], 2, dim, 16, dtype, e4m3, 23)
        good, good_lse = run_bits(cache, q, new)
        at = length - 3
        spoil(cache, "k", at, 1, 7, what)
        out, lse = run_bits(cache, q, new)
        assert same(out[:-3], good[:-3]) and same(out[:, :4], good[:, :4]), what
        assert same(lse[:-3], good_lse[:-3]) and same(lse[:, :4], good_lse[:, :4]), what
        reread(cache) if e4m3 else cache.values.update(k=f64_of(cache.k))
        page = int(cache.table[0, at // 16])
        with np.errstate(invalid="ignore"):
            score = np.einsum("thd,d->th", f64_of(q[-3:, 4:]), cache.values["k"][page, 1, at % 16])
        if e4m3 and what == "inf":      # (sum of the codes' products) * inf; the float64 products would mix signs
            codes = decode_e4m3(cache.k[page, 1, at % 16].cpu().numpy()).astype(np.float64)
            score = np.einsum("thd,d->th", f64_of(q[-3:, 4:]), codes) * math.inf
        none = torch.from_numpy(score == -math.inf).to(DEV)
        assert out[-3:, 4:][~none].isnan().all() and lse[-3:, 4:][~none].isnan().all(), what
        kk, vv = cache.request("k", 0).copy(), cache.request("v", 0)
        kk[at, 1] = 0
        for t in range(3):          # without the key, which has no weight: a request one key shorter
            if none[t].any():
                n = length - 2 + t
                keep = [j for j in range(n) if j != at]
                ref = attention_ref(f64_of(q[new - 3 + t:new - 2 + t]), kk[keep], vv[keep], len(keep) - 1, 1 / math.sqrt(dim), 0)
                pick = np.flatnonzero(np.r_[np.zeros(4, bool), none[t].cpu().numpy()])
                ref = tuple(x[:, pick] for x in ref)
                check_rows(out[new - 3 + t:new - 2 + t][:, pick], lse[new - 3 + t:new - 2 + t][:, pick], ref, dtype, n, dim, float(np.abs(vv).max()), what)


@pytest.mark.parametrize("dtype,e4m3", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("name", ["k", "v"])
def test_before_the_window_nothing_matters(name, many, dim, dtype, e4m3):
    """A key or value that no row's window reaches, in a tile of keys that some of their windows share."""
    new, window, length = few_or_many(many), 40, 230
    q = normal((new, 8, dim), dtype, 26)
    for what in ("nan", "inf", "-inf") if not e4m3 else ("nan", "inf", "code"):
        cache = Cache([length], 2, dim, 16, dtype, e4m3, 25)
        good, good_lse = run_bits(cache, q, new, window)
        spoil(cache, name, length - new - window, 1, 7, what)
        out, lse = run_bits(cache, q, new, window)
        assert same(out, good) and same(lse, good_lse), what


@pytest.mark.parametrize("dtype,e4m3", KINDS)
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_a_value_that_is_not_finite_under_a_small_weight(bad, many, dtype, e4m3):
    """A weight of e^-25 is 0 in fp16 and not in float32: the rows that see the value are not finite."""
    new, dim = few_or_many(many), 64
    q = normal((new, 8, dim), dtype, 28, 0.1) + torch.ones(dim, dtype=torch.bfloat16 if dtype == "bf16" else torch.float16, device=DEV)
    cache = Cache([150], 2, dim, 16, dtype, e4m3, 27)
    page = int(cache.table[0, 0])
    if e4m3:
        cache.k[page, :, 7], cache.ks[page, :, 7] = 0xB8, 25.0 / math.sqrt(dim)     # 0xB8: -1
    else:
        cache.k[page, :, 7] = -25.0 / math.sqrt(dim)
    good, _ = run_bits(cache, q, new)
    assert good.isfinite().all()
    spoil(cache, "v", 7, 0, 5, "code" if e4m3 and bad == "nan" else bad)
    out, _ = run_bits(cache, q, new)
    assert same(out[:, 4:], good[:, 4:])
    if bad == "nan":
        assert out[:, :4, 5].isnan().all()
    elif e4m3:
        assert not out[:, :4].isfinite().any()
    else:
        assert (out[:, :4, 5] == math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prompt_value_that_is_not_finite_under_a_small_weight(dtype):
    n, dim = 100, 128
    x = normal((n, 6, dim), dtype, 30, 0.1)
    q, k, v = x[:, :4] + 1, x[:, 4:5].clone(), x[:, 5:6].clone()
    k[7] = -25.0 / math.sqrt(dim)
    good = fp8.fp8_attn_prompt(q, k, v, cu_of([n]))
    v[7, 0, 5] = math.inf
    out = fp8.fp8_attn_prompt(q, k, v, cu_of([n]))
    assert (out[7:, :, 5] == math.inf).all() and same(out[:7], good[:7])
    rest = [c for c in range(dim) if c != 5]
    assert same(out[..., rest], good[..., rest])
