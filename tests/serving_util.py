"""Inputs, packing and the comparison shared by the tests of the serving operators."""

import numpy as np
import torch

from oracle import decode_e4m3, input_to_f32, quantize_rowwise
from oracle.serving import ROUND, attention_bound, attention_ref, lse_bound
from parity_util import DEV

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def f64_of(t):
    return t.detach().cpu().to(torch.float64).numpy()


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TORCH[dtype]).to(DEV)


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)


class Cache:
    """A paged cache holding `lens` tokens of random keys and values per request in shuffled pages;
    every place that holds no token is NaN."""

    def __init__(self, lens, heads, dim, page, dtype, e4m3, seed, spare=3, width=None, kscale=1.0):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        self.page, self.heads, self.dim, self.e4m3 = page, heads, dim, e4m3
        self.lens = list(lens)
        self.table = np.full((len(lens), width or max(1, max(need, default=1))), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        shape = (pages, heads, page, dim)
        self.used = np.zeros((pages, page), dtype=bool)
        for r, n in enumerate(lens):
            for b in range(need[r]):
                self.used[self.table[r, b], : min(page, n - b * page)] = True
        hole = torch.from_numpy(~self.used)[:, None, :, None]
        self.k, self.v, self.ks, self.vs, self.values = None, None, None, None, {}
        for name, s in (("k", kscale), ("v", 1.0)):
            g = torch.Generator().manual_seed(seed * 2 + (name == "v"))
            x = (torch.randn(shape, generator=g) * s).to(TORCH[dtype])
            if e4m3:
                q, sc = quantize_rowwise(x.view(torch.int16).numpy().view(np.uint16).reshape(-1, dim), dtype)
                vals = decode_e4m3(q).astype(np.float64) * sc.astype(np.float64)[:, None]
                self.values[name] = vals.reshape(shape)
                codes = torch.from_numpy(q.reshape(shape)).masked_fill(hole, 0x7F)
                scales = torch.from_numpy(sc.reshape(shape[:3]).copy()).masked_fill(hole[..., 0], float("nan"))
                setattr(self, name, codes.to(DEV))
                setattr(self, name + "s", scales.to(DEV))
            else:
                self.values[name] = f64_of(x)
                setattr(self, name, x.masked_fill(hole, float("nan")).to(DEV))
        self.dev_table = torch.from_numpy(self.table).to(DEV)
        self.dev_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def request(self, name, r):
        """The values [len, heads, dim] of request r, float64."""
        n = self.lens[r]
        blocks = self.table[r, : -(-n // self.page)]
        x = self.values[name][blocks].transpose(0, 2, 1, 3).reshape(-1, self.heads, self.dim)
        return x[:n]


def check_rows(out, lse, ref, dtype, keys, dim, vmax, what, rel=True):
    """One request's output rows against the oracle's, element by element, and (for normal values,
    whose rounding errors are independent) as a whole: two roundings of at most ROUND each."""
    want, want_lse, spread, size = ref
    got = f64_of(out)
    assert np.isfinite(got).all(), f"{what}: not finite"
    bound = attention_bound(want, spread, size, max(keys, 1), dim, dtype, vmax)
    off = np.abs(got - want)
    assert (off <= bound).all(), f"{what}: {(off > bound).sum()} outside, worst {np.max(off / bound):.3g} of the bound at {np.unravel_index(np.argmax(off / bound), off.shape)}"
    norm = np.linalg.norm(want)
    if rel and norm > 0 and want.size >= 256:
        assert np.linalg.norm(got - want) <= 2 * ROUND[dtype] * norm, f"{what}: rel {np.linalg.norm(got - want) / norm:.3g}"
    if lse is not None:
        g = f64_of(lse)
        some = np.isfinite(want_lse)
        assert np.array_equal(np.isneginf(g), ~some), f"{what}: rows without keys"
        assert (np.abs(g - np.where(some, want_lse, 0))[some] <= lse_bound(want_lse, size, max(keys, 1), dim)[some]).all(), f"{what}: lse"


def check_prompt(q, k, v, lens, out, lse, dtype, scale, window, rel=True):
    at = 0
    for r, n in enumerate(lens):
        s = slice(at, at + n)
        at += n
        if n:
            ref = attention_ref(f64_of(q[s]), f64_of(k[s]), f64_of(v[s]), 0, scale, window)
            check_rows(out[s], None if lse is None else lse[s], ref, dtype, n, q.shape[2], float(np.abs(f64_of(v[s])).max()), f"request {r} of {n}", rel)


def check_paged(q, cache, new, out, lse, dtype, scale, window, rel=True):
    at = 0
    for r, n in enumerate(new):
        s = slice(at, at + n)
        at += n
        if n:
            kk, vv = cache.request("k", r), cache.request("v", r)
            ref = attention_ref(f64_of(q[s]), kk, vv, len(kk) - n, scale, window)
            check_rows(out[s], None if lse is None else lse[s], ref, dtype, len(kk), q.shape[2], float(np.abs(vv).max()) if vv.size else 0.0,
                       f"request {r}: {n} new of {len(kk)}", rel)
