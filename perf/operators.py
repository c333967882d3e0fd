"""Cases of the serving operators: what one step of a batch of requests needs around the FP8 projections.

  plan    block tables, slots and positions of a step's new tokens, from the requests' lengths
  append  a step's new keys and values into a paged cache, as they are or as e4m3 codes with one scale per token and head
  prompt  causal attention over whole prompts packed one after the other, grouped heads
  paged   attention of each request's new tokens (one, or a chunk) over its pages, grouped heads

``run`` with ``own`` false computes them from elementary torch operations in float32; with ``own`` true it calls
the package.  Head counts and sizes are those of the layers in workloads.py: TinyLlama-1.1B 32 query heads on 4 of
size 64, Llama-2-7B 32 on 32 of size 128, Llama-3-8B 32 on 8 of size 128.
"""

import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # one decode step of 64 requests: every request gets one token, a few start a new page
        dict(name="plan_decode", op="plan", batch=64, page=16, longest=8000, width=512, new="one", pad=0, short=False, layout=1),
        # a step that admits prompts: 1024 requests, decode tokens and ragged prompts mixed, the token count padded up
        dict(name="plan_mixed", op="plan", batch=1024, page=64, longest=30000, width=512, new="mixed", pad=100, short=False, layout=2),
        # the keys and values of one decode step, Llama-3-8B, as e4m3
        dict(name="append_decode_e4m3", op="append", tokens=64, kv_heads=8, q_heads=32, dim=128, page=16, dtype="bf16", cache="e4m3", layout=3),
        # the keys and values of a large step of prompts, Llama-3-8B, as e4m3
        dict(name="append_prompt_e4m3", op="append", tokens=16384, kv_heads=8, q_heads=32, dim=128, page=64, dtype="bf16", cache="e4m3", layout=4),
        # the first answer to a short question, TinyLlama in fp16: latency
        dict(name="prompt_short", op="prompt", batch=1, longest=37, ragged=False, q_heads=32, kv_heads=4, dim=64, dtype="f16", window=0, lse=False, layout=5),
        # twelve prompts of very different lengths in one step, Llama-3-8B
        dict(name="prompt_packed", op="prompt", batch=12, longest=2048, ragged=True, q_heads=32, kv_heads=8, dim=128, dtype="bf16", window=0, lse=False, layout=6),
        # one long document, Llama-3-8B's heads: the largest
        dict(name="prompt_long", op="prompt", batch=1, longest=16384, ragged=False, q_heads=32, kv_heads=8, dim=128, dtype="bf16", window=0, lse=True, layout=7),
        # one user's decode step on Llama-2-7B: no heads are shared, a short context
        dict(name="decode_one", op="paged", batch=1, longest=701, ragged=False, new="one", chunk=1, q_heads=32, kv_heads=32, dim=128, page=16, dtype="bf16", cache="same", window=0, lse=False, layout=8),
        # a served batch's decode step on Llama-3-8B with an e4m3 cache
        dict(name="decode_batch_e4m3", op="paged", batch=64, longest=8192, ragged=True, new="one", chunk=1, q_heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", cache="e4m3", window=0, lse=False, layout=9),
        # four long conversations, Llama-3-8B's heads: few rows, a long axis
        dict(name="decode_long", op="paged", batch=4, longest=131072, ragged=True, new="one", chunk=1, q_heads=32, kv_heads=8, dim=128, page=64, dtype="bf16", cache="same", window=0, lse=True, layout=10),
        # prompts taken in chunks over what is cached, Llama-3-8B
        dict(name="chunk_cached", op="paged", batch=4, longest=16000, ragged=True, new="chunk", chunk=1024, q_heads=32, kv_heads=8, dim=128, page=32, dtype="bf16", cache="same", window=0, lse=False, layout=11),
        # decode tokens and chunks in one step, TinyLlama in fp16 with an e4m3 cache
        dict(name="mixed_e4m3", op="paged", batch=24, longest=2000, ragged=True, new="mixed", chunk=200, q_heads=32, kv_heads=4, dim=64, page=16, dtype="f16", cache="e4m3", window=0, lse=False, layout=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "append", "prompt", "prompt", "paged", "paged", "paged"))
    c = dict(op=op, layout=rng.randrange(1 << 30))
    page = rng.choice((16, 32, 64, 128))
    if op == "plan":
        longest = _log(rng, 1, 30000)
        return dict(c, batch=_log(rng, 1, 1024), page=page, longest=longest, width=longest // page + 2 + rng.randrange(9),
                    new=rng.choice(("one", "chunk", "mixed")), pad=rng.randrange(200), short=rng.random() < 0.2)
    kv = rng.choice((1, 2, 4, 8, 8, 32))
    heads = dict(q_heads=32 if kv == 32 else kv * rng.choice((1, 2, 4, 5, 8)), kv_heads=kv, dim=rng.choice((64, 128, 128)),
                 dtype=rng.choice(("bf16", "bf16", "f16")))
    if op == "append":
        return dict(c, tokens=_log(rng, 1, 131072 // kv), page=page, cache=rng.choice(("e4m3", "e4m3", "same")), **heads)
    c.update(heads, window=rng.choice((0, 0, 0, _log(rng, 1, 4096))), lse=rng.random() < 0.5)
    while op == "prompt":  # no more work and no larger score matrix in the plain form than prompt_long's
        c.update(batch=_log(rng, 1, 64), longest=_log(rng, 1, 16384), ragged=rng.random() < 0.7)
        if c["batch"] * c["q_heads"] * c["longest"] ** 2 <= 32 * 8192 ** 2:
            return c
    while True:
        c.update(batch=_log(rng, 1, 128), longest=_log(rng, 1, 131072), ragged=rng.random() < 0.7, new=rng.choice(("one", "one", "chunk", "mixed")),
                 page=page, cache=rng.choice(("same", "e4m3")))
        c["chunk"] = 1 if c["new"] == "one" else _log(rng, 2, 2048)
        if (c["chunk"] <= c["longest"] and c["batch"] * c["q_heads"] * c["chunk"] * c["longest"] <= 32 * 8192 ** 2
                and c["batch"] * c["longest"] * c["kv_heads"] * c["dim"] <= 4 * 131072 * 8 * 128):
            return c


# ---------------------------------------------------------------------------------------------------------------
# lengths: from the case alone


def _lens(case):
    """(cached, added) of every request, as lists."""
    r = random.Random(case["layout"])
    n, longest = case["batch"], case["longest"]
    if case["op"] == "prompt":  # a ragged batch holds a request without tokens now and then
        lens = [longest if not case["ragged"] or i == 0 else 0 if r.random() < 0.04 else _log(r, 1, longest) for i in range(n)]
        r.shuffle(lens)
        return [0] * n, lens
    cached, added = [], []
    for i in range(n):
        if case["op"] == "plan":
            total, chunk = _log(r, 1, longest), 2048
        else:
            total, chunk = longest if not case["ragged"] or i == 0 else _log(r, max(1, longest // 16), longest), case["chunk"]
        a = 1
        if case["new"] == "chunk" or (case["new"] == "mixed" and r.random() < 0.25):
            a = _log(r, 1, chunk) if case["op"] == "plan" else r.randint(max(1, chunk // 4), chunk) if i else chunk
        elif case["new"] == "mixed" and i and r.random() < 0.05:
            a = 0
        a = min(a, total)
        cached.append(total - a)
        added.append(a)
    return cached, added


def _pairs(cached, added, window):
    """Unmasked (query, key) pairs, and the keys that some query of the request sees, over all requests."""
    pairs = keys = 0
    for c, a in zip(cached, added):
        if a:
            first, last = c + 1, c + a  # keys of the first and of the last new token, before the window
            if window and window < last:
                full = max(0, min(a, window - c))  # tokens whose whole past lies in the window
                pairs += full * (2 * first + full - 1) // 2 + (a - full) * window
                keys += last - max(0, first - window)
            else:
                pairs += a * (first + last) // 2
                keys += last
    return pairs, keys


def work(case):
    if case["op"] == "append":
        n = 2 * case["tokens"] * case["kv_heads"]
        kept = case["dim"] + 4 if case["cache"] == "e4m3" else 2 * case["dim"]
        return {"bytes": n * (2 * case["dim"] + kept) + 8 * case["tokens"], "flops": n * case["dim"]}
    cached, added = _lens(case)
    tokens = sum(added)
    if case["op"] == "plan":
        page = case["page"]
        entries = sum(-(-(c + a) // page) - -(-c // page) for c, a in zip(cached, added))
        used = sum(-(-(c + a) // page) - c // page for c, a in zip(cached, added) if a)  # pages that hold a new token
        return {"bytes": 16 * len(cached) + 8 * entries + 4 * used + 12 * (tokens + case["pad"]), "flops": 0}
    pairs, keys = _pairs(cached, added, case["window"])
    row = case["kv_heads"] * (case["dim"] + 4 if case.get("cache") == "e4m3" else 2 * case["dim"])
    if case["op"] == "paged":
        row += 4 / case["page"]
    lse = 4 if case["lse"] else 0
    return {"bytes": int(tokens * case["q_heads"] * (4 * case["dim"] + lse) + 2 * keys * row), "flops": 4 * pairs * case["q_heads"] * case["dim"]}


# ---------------------------------------------------------------------------------------------------------------
# inputs


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _codes_and_scales(x):
    """Rows of x [..., D] as e4m3 values (a float8 tensor) and float32 scales [...]: amax / 448, 1 for a zero row."""
    x = x.float()
    amax = x.abs().amax(-1)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)
    return (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _rows(shape, g, dtype, spread):
    """Normal values whose channels differ in size, as projected queries, keys and values do."""
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g)
    if spread:
        x *= torch.empty(shape[-1], device="cuda").normal_(generator=g).mul_(spread).exp_()
    return x.to(dtype)


def _qkv(tokens, case, g, dtype):
    """Views of one fused projection's output [tokens, (q_heads + 2 kv_heads) dim]: rows are far apart."""
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    x = _rows((tokens, hq + 2 * hk, d), g, dtype, 0.5)
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dtype = torch.float16 if case.get("dtype") == "f16" else torch.bfloat16
    if case["op"] == "append":
        page, tokens = case["page"], case["tokens"]
        pages = -(-tokens // page) * 2 + 3
        _, s["k"], s["v"] = _qkv(tokens, case, g, dtype)
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
        if tokens > 4:  # the padding of a step that runs with a fixed token count
            s["slots"][-max(1, tokens // 64):] = -1
        shape = (pages, case["kv_heads"], page, case["dim"])
        for n in ("k", "v"):
            if case["cache"] == "e4m3":
                s[n + "_cache"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
                s[n + "_scales"] = torch.ones(shape[:3], device="cuda")
            else:
                s[n + "_cache"], s[n + "_scales"] = torch.zeros(shape, dtype=dtype, device="cuda"), None
        return s
    cached, added = _lens(case)
    s["cu"] = _ints(np.concatenate([[0], np.cumsum(added)]).tolist())
    s["tokens"], s["most"] = sum(added), max(added)
    if case["op"] == "prompt":
        s["q"], s["k"], s["v"] = _qkv(s["tokens"], case, g, dtype)
        return s
    page = case["page"]
    s["cached"], s["added"], s["lens"] = _ints(cached), _ints(added), _ints([c + a for c, a in zip(cached, added)])
    have = [-(-(c + (a if case["op"] == "paged" else 0)) // page) for c, a in zip(cached, added)]
    pages = sum(have)
    want = sum(-(-(c + a) // page) for c, a in zip(cached, added)) - pages
    order = torch.randperm(pages + want + 5, generator=g, device="cuda").int()
    width = case.get("width") or max(1, max(have))
    at = torch.arange(width, device="cuda")[None] < _ints(have)[:, None]
    s["table"] = torch.full((len(cached), width), -1, dtype=torch.int32, device="cuda")
    s["table"][at] = order[:pages]
    if case["op"] == "plan":
        s["tokens"] += case["pad"]
        s["free"] = order[pages: pages + max(1, want // 2 if case["short"] else want + 2)].contiguous()
        s["taken"] = _ints([0])
        return s
    s["longest_len"] = max(c + a for c, a in zip(cached, added))
    s["q"] = _rows((s["tokens"], case["q_heads"], case["dim"]), g, dtype, 0.0)
    shape = (pages + 5, case["kv_heads"], page, case["dim"])
    used = torch.zeros((pages + 5, page), dtype=torch.bool, device="cuda")  # the rest was never written: it may hold anything
    req, col = at.nonzero(as_tuple=True)
    used[s["table"][req, col].long()] = (col[:, None] * page + torch.arange(page, device="cuda")) < s["lens"][req][:, None]
    for n in ("k", "v"):
        x = _rows(shape, g, dtype, 0.5)
        if case["cache"] == "e4m3":
            x, scale = _codes_and_scales(x)
            s[n + "_scales"] = scale.masked_fill_(~used[:, None], math.nan)
            s[n + "_cache"] = x.view(torch.uint8).masked_fill_(~used[:, None, :, None], 0x7F)
        else:
            s[n + "_cache"], s[n + "_scales"] = x.masked_fill_(~used[:, None, :, None], math.nan), None
    return s


# ---------------------------------------------------------------------------------------------------------------
# the plain forms


def _plan(s):
    page, table, free = s["page"], s["table"], s["free"]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.cat([zero, s["added"].cumsum(0).int()])
    lens = s["cached"] + s["added"]
    old, new = (s["cached"] + page - 1) // page, (lens + page - 1) // page
    first = (new - old).cumsum(0) - (new - old)
    col = torch.arange(table.shape[1], device="cuda")
    rank = s["taken"] + first[:, None] + col[None] - old[:, None]
    fresh = (col[None] >= old[:, None]) & (col[None] < new[:, None])
    table = torch.where(fresh, torch.where(rank < free.numel(), free[rank.clamp(0, free.numel() - 1)], -1), table)
    t = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    there = t < cu[-1]
    req = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=lens.numel() - 1)
    position = torch.where(there, s["cached"][req] + t - cu[req], -1)
    block = table[req, (position // page).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(there & (block >= 0), block * page + position % page, -1)
    want = (new - old).sum().int().reshape(1)
    granted = torch.minimum(want, free.numel() - s["taken"])
    return dict(cu_tokens=cu, seq_lens=lens, positions=position, slots=slots, block_table=table, taken=s["taken"] + granted, missing=want - granted)


def _append(s):
    keep = s["slots"] >= 0
    slots = torch.where(keep, s["slots"], 0)
    block, at = slots // s["page"], slots % s["page"]
    block, at = block[keep], at[keep]
    out = {}
    for n in ("k", "v"):
        cache, scales, x = s[n + "_cache"], s[n + "_scales"], s[n][keep]
        if scales is None:
            cache[block, :, at] = x
        else:
            codes, scale = _codes_and_scales(x)
            cache[block, :, at] = codes.view(torch.uint8)
            scales[block, :, at] = scale
            out[n + "_scales"] = scales
            cache = cache.view(torch.float8_e4m3fn)
        out[n + "_cache"] = cache
    return out


def _attend(q, k, v, position, lens, scale, window):
    """q [B, Q, Hq, D], k and v [B, S, Hkv, D], float32; position [B, Q] of each query (-1: none), lens [B] of the keys."""
    b, nq, hq, d = q.shape
    hk, keys = k.shape[2], k.shape[1]
    j = torch.arange(keys, device="cuda")
    seen = (j <= position[..., None]) & (j < lens[:, None, None])
    if window:
        seen &= j > position[..., None] - window
    x = q.view(b, nq, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d) @ k.permute(0, 2, 3, 1)
    x = x.mul_(scale).view(b, hk, hq // hk, nq, keys).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    some = seen.any(-1)[:, None, None, :, None]
    o = (x.view(b, hk, -1, keys) @ v.permute(0, 2, 1, 3)).view(b, hk, hq // hk, nq, d)
    o = torch.where(some, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(b, nq, hq, d)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(b, nq, hq)
    return o, lse


def _padded(s, x, n):
    """Packed rows x [tokens, ...] as [B, n, ...], and where they are."""
    cu = s["cu"].long()
    i = torch.arange(n, device="cuda")
    there = i[None] < (cu[1:] - cu[:-1])[:, None]
    return x[(cu[:-1, None] + i[None]).clamp(max=x.shape[0] - 1)].float(), there


def _packed(o, lse, there, s):
    r = {"out": o[there].to(s["q"].dtype)}
    if s["lse"]:
        r["lse"] = lse[there]
    return r


def _prompt(s):
    n = s["most"]
    (q, there), (k, _), (v, _) = (_padded(s, s[x], n) for x in "qkv")
    position = torch.where(there, torch.arange(n, device="cuda")[None], -1)
    return _packed(*_attend(q, k, v, position, there.sum(1), 1.0 / math.sqrt(s["dim"]), s["window"]), there, s)


def _paged(s):
    q, there = _padded(s, s["q"], s["most"])
    j = torch.arange(s["longest_len"], device="cuda")
    held = j[None] < s["lens"][:, None]
    block = torch.where(held, s["table"][:, j // s["page"]], 0)
    kv = []
    for n in ("k", "v"):
        cache, scales = s[n + "_cache"], s[n + "_scales"]
        if scales is None:
            x = cache[block, :, j % s["page"]].float()
        else:
            x = cache[block, :, j % s["page"]].view(torch.float8_e4m3fn).float()
            x *= scales[block, :, j % s["page"]][..., None]
        kv.append(x.masked_fill_(~held[:, :, None, None], 0.0))
    position = torch.where(there, s["cached"][:, None] + torch.arange(s["most"], device="cuda")[None], -1)
    return _packed(*_attend(q, *kv, position, s["lens"], 1.0 / math.sqrt(s["dim"]), s["window"]), there, s)


# ---------------------------------------------------------------------------------------------------------------
# the calls


def _own(s):
    import fp8_quantized_gemm_amax_amd as fp8

    if s["op"] == "plan":
        p = fp8.fp8_paged_plan(s["cached"], s["added"], s["table"], s["free"], s["taken"], s["tokens"], s["page"])
        return dict(cu_tokens=p.cu_tokens, seq_lens=p.seq_lens, positions=p.positions, slots=p.slots, block_table=s["table"], taken=p.taken, missing=p.missing)
    if s["op"] == "append":
        fp8.fp8_kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
        if s["k_scales"] is None:
            return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
        return dict(k_scales=s["k_scales"], k_cache=s["k_cache"].view(torch.float8_e4m3fn), v_scales=s["v_scales"], v_cache=s["v_cache"].view(torch.float8_e4m3fn))
    if s["op"] == "prompt":
        r = fp8.fp8_attn_prompt(s["q"], s["k"], s["v"], s["cu"], window=s["window"], return_lse=s["lse"])
    else:
        r = fp8.fp8_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], s["k_scales"], s["v_scales"],
                               window=s["window"], max_new=s["most"], return_lse=s["lse"])
    return dict(out=r[0], lse=r[1]) if s["lse"] else dict(out=r)


def run(state):
    if own:
        return _own(state)
    return {"plan": _plan, "append": _append, "prompt": _prompt, "paged": _paged}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_rows(q, k, v, first, scale, window):
    """One request, one key head: q [n, G, D] at positions first + 0.. over k, v [S, D]; rows in pieces that fit."""
    out, lse = [], []
    step = max(1, (1 << 28) // max(1, k.shape[0] * q.shape[1]))
    j = torch.arange(k.shape[0], device="cuda")
    for i in range(0, q.shape[0], step):
        x = torch.tensordot(q[i:i + step], k, dims=([2], [1])) * scale
        p = first + torch.arange(i, i + x.shape[0], device="cuda")[:, None, None]
        x[((j > p) | ((j <= p - window) if window else (j < 0))).expand_as(x)] = -math.inf
        z = torch.logsumexp(x, -1)
        out.append(torch.tensordot(torch.exp(x - z[..., None]), v, dims=([2], [0])))
        lse.append(z)
    return torch.cat(out), torch.cat(lse)


def _e4m3_grid():
    """All finite e4m3 magnitudes in rising order."""
    tiny = [m / 512.0 for m in range(8)]
    return np.array(tiny + [(1 + m / 8.0) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1])


def _exact_append(s):
    """The codes' values and scales, from amax / 448 in float64 and the nearest grid value (ties to the even code)."""
    grid = torch.from_numpy(_e4m3_grid()).cuda()
    half = (grid[1:] + grid[:-1]) / 2
    out = {}
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    for n in ("k", "v"):
        x, cache = s[n][keep].double(), s[n + "_cache"].double() if s["cache"] == "same" else torch.zeros(s[n + "_cache"].shape, dtype=torch.float64, device="cuda")
        if s["cache"] == "e4m3":
            scale = x.abs().amax(-1) / E4M3_MAX
            scale[scale == 0] = 1.0
            y = x / scale[..., None]
            at = torch.bucketize(y.abs(), half)  # how many midpoints lie below |y|
            at += ((at < half.numel()) & (half[at.clamp(max=half.numel() - 1)] == y.abs()) & (at % 2 == 1)).long()
            x = torch.copysign(grid[at], y)
            scales = torch.ones(cache.shape[:3], dtype=torch.float64, device="cuda")
            scales[slots // s["page"], :, slots % s["page"]] = scale
            out[n + "_scales"] = scales
        cache[slots // s["page"], :, slots % s["page"]] = x
        out[n + "_cache"] = cache
    return out


def _exact_plan(s):
    page, free = s["page"], s["free"].tolist()
    table, slots, positions, cu, lens, used, missing = s["table"].cpu().numpy().copy(), [], [], [0], [], int(s["taken"]), 0
    for i, (c, a) in enumerate(zip(s["cached"].tolist(), s["added"].tolist())):
        for t in range(c, c + a):
            if t % page == 0:
                table[i, t // page] = free[used] if used < len(free) else -1
                missing += used >= len(free)
                used += used < len(free)
            positions.append(t)
            slots.append(int(table[i, t // page]) * page + t % page if table[i, t // page] >= 0 else -1)
        cu.append(cu[-1] + a)
        lens.append(c + a)
    rest = [-1] * (s["tokens"] - len(slots))
    return dict(cu_tokens=np.array(cu), seq_lens=np.array(lens), positions=np.array(positions + rest), slots=np.array(slots + rest),
                block_table=table, taken=np.array([used]), missing=np.array([missing]))


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "plan":
        return _exact_plan(s)
    if s["op"] == "append":
        return _exact_append(s)
    cu, hk, group = s["cu"].tolist(), s["kv_heads"], s["q_heads"] // s["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if a == b:
            continue
        n = b - a if s["op"] == "prompt" else int(s["lens"][i])
        for h in range(hk):
            if s["op"] == "prompt":
                k, v = (s[x][a:b, h].double() for x in "kv")
            else:
                blocks = s["table"][i, : -(-n // s["page"])].long()
                kv = []
                for x in ("k", "v"):
                    y = s[x + "_cache"][blocks, h]
                    y = y.double() if s["cache"] == "same" else y.view(torch.float8_e4m3fn).double() * s[x + "_scales"][blocks, h].double()[..., None]
                    kv.append(y.reshape(-1, y.shape[-1])[:n])
                k, v = kv
            heads = slice(h * group, (h + 1) * group)
            o, z = _exact_rows(s["q"][a:b, heads].double(), k, v, n - (b - a), 1.0 / math.sqrt(s["dim"]), s["window"])
            out[a:b, heads], lse[a:b, heads] = o, z
    return dict(out=out, lse=lse) if s["lse"] else dict(out=out)
