"""A served attention block: FP8 projections, a paged e4m3 key/value cache and attention, for
requests that come and go.

    python examples/serve_attention.py

Each step takes the new tokens of all running requests at once (whole prompts, chunks of long
ones, single tokens): the plan hands out pages and slots on the GPU from the requests' lengths,
the fused QKV projection runs as an FP8 GEMM with 1x128 activation scales, the new keys and
values go into their pages as e4m3 with one scale per token and head, attention reads the pages,
and the output projection is an FP8 GEMM again.  Lengths stay on the GPU; the host knows how
many tokens a step has and never waits.  At the end every request's last output is compared with
the same tokens run as one whole prompt (fp8_attn_prompt on unquantized keys and values).
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_quantized_gemm_amax_amd as fp8   # noqa: E402


class AttentionBlock:
    """Projections with random weights, quantized once in 128x128 blocks."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, device, seed=0):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            w = torch.empty((n, k), device=device).normal_(0, k ** -0.5, generator=g).bfloat16()
            return fp8.fp8_quantize_per_token_group(w, 128, 128)

        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, q_heads * head_dim)

    @staticmethod
    def project(x, weight):
        q, s = fp8.fp8_quantize_per_token_group(x, 1, 128)
        return fp8.fp8_gemm_scaled_blockwise(q, s, *weight)

    def heads(self, x):
        """q, k and v of x [tokens, hidden]: views of the fused projection's output."""
        y = self.project(x, self.qkv).view(x.shape[0], -1, self.head_dim)
        return y.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)

    def step(self, x, plan, cache, max_new):
        q, k, v = self.heads(x)
        fp8.fp8_kv_append(k, v, plan.slots, cache.k, cache.v, cache.k_scales, cache.v_scales)
        a = fp8.fp8_attn_paged(q, cache.k, cache.v, cache.table, plan.seq_lens, plan.cu_tokens,
                               cache.k_scales, cache.v_scales, max_new=max_new)
        return self.project(a.view(x.shape[0], -1), self.out)

    def whole(self, x, cu_tokens):
        """The same for whole prompts, without a cache."""
        a = fp8.fp8_attn_prompt(*self.heads(x), cu_tokens)
        return self.project(a.view(x.shape[0], -1), self.out)


class PagedCache:
    """The pages, and the batch's tables and lengths, all on the GPU."""

    def __init__(self, pages, page_size, requests, width, block, device):
        shape = (pages, block.kv_heads, page_size, block.head_dim)
        self.page_size = page_size
        self.k, self.v = (torch.empty(shape, dtype=torch.uint8, device=device) for _ in "kv")
        self.k_scales, self.v_scales = (torch.empty(shape[:3], device=device) for _ in "kv")
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.free = torch.randperm(pages, device=device).int()
        self.taken = torch.zeros(1, dtype=torch.int32, device=device)

    def plan(self, added, tokens):
        plan = fp8.fp8_paged_plan(self.lens, added, self.table, self.free, self.taken, tokens, self.page_size)
        self.lens, self.taken = plan.seq_lens, plan.taken
        return plan


def serve(prompts=(37, 300, 5, 129), chunk=96, answers=6, hidden=1024, q_heads=16, kv_heads=4, head_dim=64, seed=0):
    """Runs the requests to the end; returns the largest relative difference of a request's last
    output from the whole-prompt run, and the number of steps."""
    device = torch.device("cuda:0")
    block = AttentionBlock(hidden, q_heads, kv_heads, head_dim, device, seed)
    cache = PagedCache(64, 16, len(prompts), 32, block, device)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    totals = [n + answers for n in prompts]
    tokens = [torch.empty((n, hidden), device=device).normal_(generator=g).bfloat16() for n in totals]
    done, last, steps, missing = [0] * len(prompts), {}, 0, torch.zeros(1, dtype=torch.int32, device=device)
    while any(d < n for d, n in zip(done, totals)):
        # a prompt's next chunk, or one token of the answer; finished requests bring nothing
        new = [min(chunk, p - d) if d < p else min(1, n - d) for p, d, n in zip(prompts, done, totals)]
        x = torch.cat([t[d:d + a] for t, d, a in zip(tokens, done, new)])
        plan = cache.plan(torch.tensor(new, dtype=torch.int32, device=device), x.shape[0])
        y = block.step(x, plan, cache, max(new))
        missing |= plan.missing
        at = 0
        for r, a in enumerate(new):
            at += a
            done[r] += a
            if a:
                last[r] = y[at - 1]
        steps += 1
    assert int(missing) == 0, "the cache ran out of pages"
    cu = torch.tensor([0] + totals, dtype=torch.int32, device=device).cumsum(0).int()
    want = block.whole(torch.cat(tokens), cu)
    ends = [sum(totals[:i + 1]) - 1 for i in range(len(totals))]
    off = max(float((last[r].float() - want[e].float()).norm() / want[e].float().norm()) for r, e in enumerate(ends))
    return off, steps


if __name__ == "__main__":
    off, steps = serve()
    print(f"{steps} steps; the last outputs differ from whole prompts by {off:.2%} (e4m3 keys and values)")
