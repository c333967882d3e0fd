"""A paged cache in four bits for the tests, with the interface of serving_util.Cache."""

import numpy as np
import torch

from oracle import mxfp4
from parity_util import DEV


class Cache4:
    """`lens` tokens of random codes and scales per request in shuffled pages; every place that holds
    no token has codes 0xFF and the scale byte of NaN.  `low`, `high`: the scale bytes' range."""

    def __init__(self, lens, heads, dim, page, seed, spare=3, width=None, low=124, high=127):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        self.page, self.heads, self.dim, self.lens = page, heads, dim, list(lens)
        self.table = np.full((len(lens), width or max(1, max(need, default=1))), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        used = np.zeros((pages, page), dtype=bool)
        for r, n in enumerate(lens):
            for b in range(need[r]):
                used[self.table[r, b], : min(page, n - b * page)] = True
        hole = ~used[:, None, :, None]
        self.values = {}
        for name in "kv":
            codes = np.where(hole, 0xFF, rng.integers(0, 256, (pages, heads, page, dim // 2))).astype(np.uint8)
            scales = np.where(hole, 255, rng.integers(low, high + 1, (pages, heads, page, dim // 32))).astype(np.uint8)
            setattr(self, name, torch.from_numpy(codes).to(DEV))
            setattr(self, name + "s", torch.from_numpy(scales).to(DEV))
        self.reread()
        self.dev_table = torch.from_numpy(self.table).to(DEV)
        self.dev_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def reread(self):
        """The values from what the tensors hold now."""
        for name in "kv":
            self.values[name] = mxfp4.decode(getattr(self, name).cpu().numpy(), getattr(self, name + "s").cpu().numpy())

    def request(self, name, r):
        """The values [len, heads, dim] of request r, float64."""
        n = self.lens[r]
        blocks = self.table[r, : -(-n // self.page)]
        x = self.values[name][blocks].transpose(0, 2, 1, 3).reshape(-1, self.heads, self.dim)
        return x[:n]

    def place(self, r, token):
        return int(self.table[r, token // self.page]), token % self.page
