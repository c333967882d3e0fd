"""Cases of the operators around a served attention block in few bits.

  rope    rotation of a step's new queries and keys by their positions, and the write of keys and values into a paged cache
  paged4  attention of each request's new tokens over a paged cache held in 4 bits (e2m1 codes, a power-of-two scale for
          every 32 channels)
  quant8  a matrix as 8-bit integers with one scale a row (a token, or an output channel)
  gemm8   the product of two such matrices

``run`` with ``own`` false computes them from elementary torch operations in float32 (float64 for the quotients of quant8,
which lie next to borders); with ``own`` true it calls the package.  Head counts and sizes are those of the layers in
workloads.py: TinyLlama-1.1B 32 query heads on 4 of size 64, hidden size 2048; Llama-2-7B 32 on 32 of size 128, 4096 and
11008; Llama-3-8B 32 on 8 of size 128, 4096 and 14336.
"""

import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decode step of 64 requests, Llama-3-8B, into an e4m3 cache: latency
        dict(name="rope_decode_e4m3", op="rope", tokens=64, q_heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False, page=16, dtype="bf16", cache="e4m3", longest=8192, chunk=1, layout=1),
        # a ragged step of chunks, TinyLlama's heads in fp16, half of the channels rotated in neighbouring pairs, a 16-bit cache
        dict(name="rope_chunks_f16", op="rope", tokens=1237, q_heads=32, kv_heads=4, dim=64, rotary=32, interleaved=True, page=32, dtype="f16", cache="same", longest=2048, chunk=300, layout=2),
        # a large step of prompts, Llama-3-8B, into an e4m3 cache
        dict(name="rope_prompt_e4m3", op="rope", tokens=16384, q_heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False, page=64, dtype="bf16", cache="e4m3", longest=8192, chunk=4096, layout=4),
        # one user's decode step, TinyLlama in fp16: latency
        dict(name="attn4_one", op="paged4", batch=1, longest=701, ragged=False, new="one", chunk=1, q_heads=32, kv_heads=4, dim=64, page=16, dtype="f16", window=0, lse=False, layout=5),
        # a served batch's decode step on Llama-3-8B
        dict(name="attn4_batch", op="paged4", batch=64, longest=8192, ragged=True, new="one", chunk=1, q_heads=32, kv_heads=8, dim=128, page=16, dtype="bf16", window=0, lse=False, layout=6),
        # four long conversations, Llama-3-8B's heads: few rows, a long axis
        dict(name="attn4_long", op="paged4", batch=4, longest=131072, ragged=True, new="one", chunk=1, q_heads=32, kv_heads=8, dim=128, page=64, dtype="bf16", window=0, lse=True, layout=7),
        # prompts taken in chunks over what is cached, Llama-3-8B
        dict(name="attn4_chunk", op="paged4", batch=4, longest=16000, ragged=True, new="chunk", chunk=1024, q_heads=32, kv_heads=8, dim=128, page=32, dtype="bf16", window=0, lse=False, layout=8),
        # the activations of a small batch before a projection of Llama-2-7B: latency
        dict(name="quant8_decode", op="quant8", rows=16, cols=4096, dtype="bf16"),
        # the activations of a large step before Llama-3-8B's down-projection
        dict(name="quant8_prefill", op="quant8", rows=4096, cols=14336, dtype="bf16"),
        # one token through Llama-2-7B's up-projection
        dict(name="gemm8_one", op="gemm8", m=1, n=11008, k=4096, dtype="bf16"),
        # a ragged batch of decode tokens through TinyLlama's up-projection, fp16 outputs
        dict(name="gemm8_batch", op="gemm8", m=61, n=5632, k=2048, dtype="f16"),
        # a large step of prompts through Llama-3-8B's up-projection
        dict(name="gemm8_prefill", op="gemm8", m=4096, n=14336, k=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "rope", "paged4", "paged4", "paged4", "quant8", "gemm8", "gemm8"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if op == "quant8":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 1, 14336 // 8) * 8 + rng.choice((0, 0, 0, 3)), dtype=dtype)
            if c["rows"] * c["cols"] <= 4096 * 14336:
                return c
    if op == "gemm8":
        while True:
            c = dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 1, 16384), k=_log(rng, 1, 14336 // 16) * 16, dtype=dtype)
            if c["m"] * c["n"] * c["k"] <= 4096 * 14336 * 4096:
                return c
    kv = rng.choice((1, 2, 4, 8, 8, 32))
    c = dict(op=op, layout=rng.randrange(1 << 30), page=rng.choice((16, 32, 64, 128)), q_heads=32 if kv == 32 else kv * rng.choice((1, 2, 4, 5, 8)),
             kv_heads=kv, dim=rng.choice((64, 128, 128)), dtype=dtype)
    if op == "rope":
        longest = _log(rng, 16, 131072)
        most = 16384 * 48 // (c["q_heads"] + 2 * kv)   # heads to move: no more than rope_prompt_e4m3's
        return dict(c, tokens=_log(rng, 1, most), rotary=rng.choice((c["dim"], c["dim"], c["dim"] // 2, 48)), interleaved=rng.random() < 0.3,
                    cache=rng.choice(("e4m3", "e4m3", "same")), longest=longest, chunk=rng.choice((1, _log(rng, 1, longest))))
    c.update(window=rng.choice((0, 0, 0, _log(rng, 1, 4096))), lse=rng.random() < 0.5)
    while True:  # no more scores than attn4_chunk's plain form can hold, no larger cache than attn4_long's
        c.update(batch=_log(rng, 1, 128), longest=_log(rng, 1, 131072), ragged=rng.random() < 0.7, new=rng.choice(("one", "one", "chunk", "mixed")))
        c["chunk"] = 1 if c["new"] == "one" else _log(rng, 2, 2048)
        if (c["chunk"] <= c["longest"] and c["batch"] * c["q_heads"] * c["chunk"] * c["longest"] <= 32 * 8192 ** 2
                and c["batch"] * c["longest"] * c["kv_heads"] * c["dim"] <= 4 * 131072 * 8 * 128):
            return c


# ---------------------------------------------------------------------------------------------------------------
# lengths: from the case alone


def _positions(case):
    """The positions of a rotation step's tokens: runs of up to `chunk` of each request, at the end of what it has."""
    r, out = random.Random(case["layout"]), []
    while len(out) < case["tokens"]:
        n = min(r.randint(max(1, case["chunk"] // 2), case["chunk"]), case["tokens"] - len(out))
        last = r.randint(n, max(n, case["longest"]))
        out.extend(range(last - n, last))
    return out


def _lens(case):
    """(cached, added) of every request, as lists."""
    r = random.Random(case["layout"])
    longest, chunk = case["longest"], case["chunk"]
    cached, added = [], []
    for i in range(case["batch"]):
        total = longest if not case["ragged"] or i == 0 else _log(r, max(1, longest // 16), longest)
        a = 1
        if case["new"] == "chunk" or (case["new"] == "mixed" and r.random() < 0.25):
            a = r.randint(max(1, chunk // 4), chunk) if i else chunk
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
        if not a:
            continue
        if window:
            pairs += sum(min(p, window) for p in range(c + 1, c + a + 1))
            keys += c + a - max(0, c + 1 - window)
        else:
            pairs += a * (2 * c + a + 1) // 2
            keys += c + a
    return pairs, keys


def work(case):
    if case["op"] == "quant8":
        n = case["rows"] * case["cols"]
        return {"bytes": 3 * n + 4 * case["rows"], "flops": 2 * n}
    if case["op"] == "gemm8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + 2 * m * n, "flops": 2 * m * n * k}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        t = case["tokens"]
        kept = d + 4 if case["cache"] == "e4m3" else 2 * d
        rows = len(set(_positions(case)))
        return {"bytes": t * (4 * d * hq + 2 * hk * (2 * d + kept) + 12) + 4 * rows * case["rotary"], "flops": t * (hq + hk) * case["rotary"] * 3}
    cached, added = _lens(case)
    pairs, keys = _pairs(cached, added, case["window"])
    row = hk * (d // 2 + d // 32)
    return {"bytes": int(sum(added) * hq * (4 * d + (4 if case["lse"] else 0)) + 2 * keys * row + 4 * keys / case["page"]), "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------------------------------------------
# inputs


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _rows(shape, g, dtype, spread):
    """Normal values whose channels differ in size, as projected queries, keys and values do."""
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g)
    if spread:
        x *= torch.empty(shape[-1], device="cuda").normal_(generator=g).mul_(spread).exp_()
    return x.to(dtype)


def _to_fp4(x):
    """x [..., D] float32 as packed e2m1 codes uint8 [..., D / 2] (an even channel in the low half of a byte) and scale
    bytes uint8 [..., D / 32]: 2^(byte - 127) is the smallest power of two not below amax / 6."""
    b = x.unflatten(-1, (-1, 32))
    mant, exp = torch.frexp(b.abs().amax(-1))     # amax = mant 2^exp, 0.5 <= mant < 1: amax / 6 <= 2^(exp - 3 + (mant > 0.75))
    e = torch.where(mant == 0, 0, exp - 3 + (mant > 0.75).int())
    y = torch.ldexp(b, -e[..., None])
    a = y.abs()
    code = torch.zeros(a.shape, dtype=torch.uint8, device=x.device)
    for at, tie in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= at) if tie else (a > at)    # ties to the even code
    code += (y < 0).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dtype = torch.float16 if case["dtype"] == "f16" else torch.bfloat16
    s["type"] = dtype
    if case["op"] == "quant8":
        s["x"] = _rows((case["rows"], case["cols"]), g, dtype, 1.0)
        return s
    if case["op"] == "gemm8":  # operands as a quantizer leaves them: a row's largest magnitude is 127
        for n, rows, spread in (("a", case["m"], 0.5), ("b", case["n"], 0.0)):
            x = _rows((rows, case["k"]), g, torch.float32, spread)
            scale = x.abs().amax(1) / 127
            s["q" + n], s["s" + n] = (x / scale[:, None]).round_().to(torch.int8), scale * (1.0 if n == "a" else 0.02)
        return s
    hq, hk, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "rope":
        tokens = case["tokens"]
        x = _rows((tokens, hq + 2 * hk, d), g, dtype, 0.5)   # views of one fused projection's output
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        half = case["rotary"] // 2
        angle = torch.arange(case["longest"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = _ints(_positions(case))
        pages = -(-tokens // page) * 2 + 3
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
        if tokens > 4:  # the padding of a step that runs with a fixed token count
            s["slots"][-max(1, tokens // 64):] = -1
            s["positions"][-max(1, tokens // 64):] = -1
        shape = (pages, hk, page, d)
        for n in "kv":
            if case["cache"] == "e4m3":
                s[n + "_cache"], s[n + "_scales"] = torch.zeros(shape, dtype=torch.uint8, device="cuda"), torch.ones(shape[:3], device="cuda")
            else:
                s[n + "_cache"], s[n + "_scales"] = torch.zeros(shape, dtype=dtype, device="cuda"), None
        s["out"] = torch.zeros((tokens, hq, d), dtype=dtype, device="cuda")  # rows of the padding stay as they are
        return s
    cached, added = _lens(case)
    s["cu"] = _ints(np.concatenate([[0], np.cumsum(added)]).tolist())
    s["tokens"], s["most"], s["longest_len"] = sum(added), max(added), max(c + a for c, a in zip(cached, added))
    s["cached"], s["lens"] = _ints(cached), _ints([c + a for c, a in zip(cached, added)])
    have = [-(-(c + a) // page) for c, a in zip(cached, added)]
    pages = sum(have)
    order = torch.randperm(pages + 5, generator=g, device="cuda").int()
    at = torch.arange(max(1, max(have)), device="cuda")[None] < _ints(have)[:, None]
    s["table"] = torch.full(at.shape, -1, dtype=torch.int32, device="cuda")
    s["table"][at] = order[:pages]
    s["q"] = _rows((s["tokens"], hq, d), g, dtype, 0.0)
    used = torch.zeros((pages + 5, page), dtype=torch.bool, device="cuda")  # the rest was never written: it may hold anything
    req, col = at.nonzero(as_tuple=True)
    used[s["table"][req, col].long()] = (col[:, None] * page + torch.arange(page, device="cuda")) < s["lens"][req][:, None]
    for n in "kv":
        codes, scales = _to_fp4(_rows((pages + 5, hk, page, d), g, torch.float32, 0.5))
        s[n + "_cache"] = codes.masked_fill_(~used[:, None, :, None], 0x77)
        s[n + "_scales"] = scales.masked_fill_(~used[:, None, :, None], 255)   # NaN
    return s


# ---------------------------------------------------------------------------------------------------------------
# the plain forms


def _rotated(x, positions, s):
    """x [tokens, heads, D] in float32, rotated by the table's rows."""
    r, half = s["rotary"], s["rotary"] // 2
    x = x.float()
    row = s["cos_sin"][positions][:, None]
    cos, sin = row[..., :half], row[..., half:]
    if s["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1) if r < x.shape[-1] else y


def _rope(s):
    keep = s["positions"] >= 0
    s["out"][keep] = _rotated(s["q"][keep], s["positions"][keep], s).to(s["type"])
    slots = s["slots"][keep]
    block, at = slots // s["page"], slots % s["page"]
    out = dict(q=s["out"])
    for n, x in (("k", _rotated(s["k"][keep], s["positions"][keep], s)), ("v", s["v"][keep].float())):
        cache, scales = s[n + "_cache"], s[n + "_scales"]
        if scales is None:
            cache[block, :, at] = x.to(s["type"])
        else:
            amax = x.abs().amax(-1)
            scale = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)
            cache[block, :, at] = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
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


def _paged4(s):
    cu = s["cu"].long()
    i = torch.arange(s["most"], device="cuda")
    there = i[None] < (cu[1:] - cu[:-1])[:, None]
    q = s["q"][(cu[:-1, None] + i[None]).clamp(max=s["tokens"] - 1)].float()
    j = torch.arange(s["longest_len"], device="cuda")
    held = j[None] < s["lens"][:, None]
    block = torch.where(held, s["table"][:, j // s["page"]], 0)
    values = torch.tensor(FP4 + tuple(-x for x in FP4), device="cuda")
    kv = []
    for n in "kv":
        c = s[n + "_cache"][block, :, j % s["page"]]
        x = values[torch.stack([c & 15, c >> 4], -1).flatten(-2).int()]
        scale = torch.exp2(s[n + "_scales"][block, :, j % s["page"]].float() - 127)
        x = (x.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)
        kv.append(x.masked_fill_(~held[:, :, None, None], 0.0))
    position = torch.where(there, s["cached"][:, None] + i[None], -1)
    o, lse = _attend(q, *kv, position, s["lens"], 1.0 / math.sqrt(s["dim"]), s["window"])
    r = dict(out=o[there].to(s["type"]))
    if s["lse"]:
        r["lse"] = lse[there]
    return r


def _quant8(s):
    x = s["x"].float()
    amax = x.abs().amax(1)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / 127)
    return dict(q=(x.double() / scale[:, None].double()).round_().to(torch.int8), scales=scale)


def _gemm8(s):
    return dict(out=(s["qa"].float() @ s["qb"].float().T * s["sa"][:, None] * s["sb"]).to(s["type"]))


# ---------------------------------------------------------------------------------------------------------------
# the calls


def _own(s):
    import fp8_quantized_gemm_amax_amd as fp8

    if s["op"] == "rope":
        fp8.fp8_rope_append(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                            interleaved=s["interleaved"], out=s["out"])
        if s["k_scales"] is None:
            return dict(q=s["out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
        return dict(q=s["out"], k_scales=s["k_scales"], k_cache=s["k_cache"].view(torch.float8_e4m3fn), v_scales=s["v_scales"],
                    v_cache=s["v_cache"].view(torch.float8_e4m3fn))
    if s["op"] == "paged4":
        r = fp8.fp8_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], s["k_scales"], s["v_scales"],
                               window=s["window"], max_new=s["most"], return_lse=s["lse"])
        return dict(out=r[0], lse=r[1]) if s["lse"] else dict(out=r)
    if s["op"] == "quant8":
        q, scales = fp8.int8_quantize_rowwise(s["x"])
        return dict(q=q, scales=scales)
    return dict(out=fp8.int8_gemm_scaled_rowwise(s["qa"], s["sa"], s["qb"], s["sb"], out_dtype=s["type"]))


def run(state):
    if own:
        return _own(state)
    return {"rope": _rope, "paged4": _paged4, "quant8": _quant8, "gemm8": _gemm8}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_rope(s):
    """Pairs as complex numbers; codes as the nearest of all e4m3 values (ties to the even code)."""
    grid = np.array([m / 512.0 for m in range(8)] + [(1 + m / 8.0) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1])
    grid = torch.from_numpy(grid).cuda()
    half = (grid[1:] + grid[:-1]) / 2
    r, n = s["rotary"], s["rotary"] // 2
    first = torch.arange(n, device="cuda") * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else n)
    kept = (s["positions"] >= 0).nonzero()[:, 0]
    turn = s["cos_sin"].double()[s["positions"][kept].long()]
    turn = torch.complex(turn[:, :n], turn[:, n:])[:, None]

    def rotate(x):
        x = x[kept].double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    q[kept] = rotate(s["q"])
    out = dict(q=q)
    slots = s["slots"][kept]
    for name, x in (("k", rotate(s["k"])), ("v", s["v"][kept].double())):
        cache = torch.zeros(s[name + "_cache"].shape, dtype=torch.float64, device="cuda")
        if s["cache"] == "e4m3":
            scale = x.abs().amax(-1) / E4M3_MAX
            scale[scale == 0] = 1.0
            y = x / scale[..., None]
            at = torch.bucketize(y.abs(), half)  # how many midpoints lie below |y|
            at += ((at < half.numel()) & (half[at.clamp(max=half.numel() - 1)] == y.abs()) & (at % 2 == 1)).long()
            x = torch.copysign(grid[at], y)
            scales = torch.ones(cache.shape[:3], dtype=torch.float64, device="cuda")
            scales[slots // s["page"], :, slots % s["page"]] = scale
            out[name + "_scales"] = scales
        cache[slots // s["page"], :, slots % s["page"]] = x
        out[name + "_cache"] = cache
    return out


def _fp4_value(codes):
    """The numbers of e2m1 codes: sign, two bits of exponent (bias 1), one of mantissa."""
    e, m = ((codes >> 1) & 3).double(), (codes & 1).double()
    x = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
    return torch.where(codes >= 8, -x, x)


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


def _exact_paged4(s):
    cu, hk, group = s["cu"].tolist(), s["kv_heads"], s["q_heads"] // s["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if a == b:
            continue
        n = int(s["lens"][i])
        blocks = s["table"][i, : -(-n // s["page"])].long()
        for h in range(hk):
            kv = []
            for x in "kv":
                c = s[x + "_cache"][blocks, h].reshape(-1, s["dim"] // 2)[:n]
                y = torch.empty((n, s["dim"]), dtype=torch.float64, device="cuda")
                y[:, 0::2], y[:, 1::2] = _fp4_value(c & 15), _fp4_value(c >> 4)
                power = s[x + "_scales"][blocks, h].reshape(-1, s["dim"] // 32)[:n].double() - 127
                kv.append(y * torch.exp2(power).repeat_interleave(32, 1))
            heads = slice(h * group, (h + 1) * group)
            out[a:b, heads], lse[a:b, heads] = _exact_rows(s["q"][a:b, heads].double(), *kv, n - (b - a), 1.0 / math.sqrt(s["dim"]), s["window"])
    return dict(out=out, lse=lse) if s["lse"] else dict(out=out)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        return _exact_rope(s)
    if s["op"] == "paged4":
        return _exact_paged4(s)
    if s["op"] == "quant8":  # the scale is the float32 number nearest to amax / 127, the code the integer nearest to x / scale
        top = s["x"].abs().amax(1).double()
        scale = torch.where(top == 0, 1.0, top / 127).float()
        low = torch.floor(s["x"].double() / scale.double()[:, None])
        over = s["x"].double() - (low + 0.5) * scale.double()[:, None]   # exact: 33 bits
        return dict(q=(low + ((over > 0) | ((over == 0) & (low % 2 != 0))).double()).to(torch.int8), scales=torch.where(top == 0, 1.0, top / 127))
    return dict(out=torch.mm(s["qa"].double(), s["qb"].double().T) * (s["sa"].double()[:, None] * s["sb"].double()[None, :]))
