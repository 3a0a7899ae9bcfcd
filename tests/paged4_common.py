"""Inputs shared by the tests of the 4-bit cache."""
from __future__ import annotations

import numpy as np

from oracle import paged as opaged
from oracle import paged4 as opaged4
from paged_common import bf16, i32


class Cache4:
    """A pool on the host (packed codes, block scales, exponents, bounds) and its copy on
    the GPU."""

    def __init__(self, seed, pages, heads, P, D, layout="heads", exps=True):
        rng = np.random.default_rng(seed)
        self.pages, self.heads, self.P, self.D, self.layout = pages, heads, P, D, layout
        self.codes, self.scales = [], []
        for _ in "kv":
            x = rng.standard_normal((pages * P, heads, D)) * np.exp2(rng.integers(-2, 3, (pages * P, heads, 1)))
            c, s = opaged4.quantise(opaged.bf16_round(x), np.zeros(heads))
            self.codes.append(np.ascontiguousarray(c.reshape(pages, P, heads, D // 2).swapaxes(1, 2)))
            self.scales.append(np.ascontiguousarray(s.reshape(pages, P, heads, D // 16).swapaxes(1, 2)))
        self.exps = [rng.integers(-3, 4, heads) if exps else None for _ in "kv"]
        b = np.sort(rng.standard_normal((pages, heads, 2, D)) * 2, axis=2)[:, :, ::-1]
        self.bounds = opaged.bf16_round(b)

    def values(self, side):
        return opaged4.values(self.codes[side], self.scales[side], self.exps[side])

    def to(self, dev, bounds=True):
        import torch
        from sparse_mla_decode_gb300 import binding
        t = []
        for c in self.codes:
            if self.layout == "tokens":
                t.append(torch.from_numpy(np.ascontiguousarray(c.swapaxes(1, 2))).to(dev).transpose(1, 2))
            else:
                t.append(torch.from_numpy(c).to(dev))
        if self.layout == "paired":  # both sides of a page in one allocation
            both = torch.stack(t, 1)
            t = [both[:, 0], both[:, 1]]
        s = [torch.from_numpy(x).to(dev) for x in self.scales]
        e = [None if x is None else i32(x, dev) for x in self.exps]
        return binding.PagedCache4(t[0], t[1], s[0], s[1], e[0], e[1], bf16(self.bounds, dev) if bounds else None)

    def attend(self, q, table, lengths, G=1, lists=None, counts=None, sm_scale=None):
        return opaged4.attend(q, self.values(0), self.values(1), table, lengths,
                              self.D ** -0.5 if sm_scale is None else sm_scale, G, lists, counts)
