"""Inputs and comparisons shared by the paged-cache tests."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np

from oracle import paged as opaged

TESTS = os.path.dirname(os.path.abspath(__file__))


class Cache:
    """A pool on the host (codes, scales, bounds) and its copy on the GPU."""

    def __init__(self, seed, pages, heads, P, D, layout="heads"):
        rng = np.random.default_rng(seed)
        self.pages, self.heads, self.P, self.D = pages, heads, P, D
        self.codes = [opaged.e4m3_encode(rng.standard_normal((pages, heads, P, D)) * 100)
                      for _ in "kv"]
        self.scales = [np.exp2(rng.integers(-9, -5, (pages, heads))).astype(np.float32)
                       for _ in "kv"]
        b = np.sort(rng.standard_normal((pages, heads, 2, D)) * 2, axis=2)[:, :, ::-1]
        self.bounds = opaged.bf16_round(b)
        self.layout = layout

    def values(self, side):
        return opaged.VALUES[self.codes[side]] * self.scales[side][..., None, None]

    def to(self, dev):
        import torch
        from sparse_mla_decode_gb300 import binding
        t = []
        for c in self.codes:
            if self.layout == "heads":
                t.append(torch.from_numpy(c).to(dev))
            elif self.layout == "tokens":
                t.append(torch.from_numpy(np.ascontiguousarray(c.swapaxes(1, 2))).to(dev).transpose(1, 2))
            else:  # both sides of a page in one allocation
                t.append(torch.from_numpy(c))
        if self.layout == "paired":
            both = torch.stack(t, 1).to(dev)  # [pages, 2, heads, P, D]
            t = [both[:, 0], both[:, 1]]
        s = [torch.from_numpy(x).to(dev) for x in self.scales]
        return binding.PagedCache(t[0], t[1], s[0], s[1], bf16(self.bounds, dev))


def bf16(x, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dev).bfloat16()


def i32(x, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)


def table_for(rng, lengths, P, pages, extra=0):
    """A table of distinct random pages; entries past a length name no page of the pool."""
    need = [-(-n // P) for n in lengths]
    W = max(max(need, default=0), 1) + extra
    free = list(rng.permutation(pages))
    table = np.full((len(lengths), W), 2 ** 30, dtype=np.int32)
    for r, n in enumerate(need):
        for j in range(n):
            table[r, j] = free.pop()
    return table


def tolerances(ref, reach, spread, lse):
    """What separates the kernel from 64 bits. A logit's fp32 sum over up to 256
    columns in steps of 16, each step rounding (or cutting) at 2^-22 of sums that
    stay below `reach`, and the scaling after it: 2^-17 reach. A weight: e to
    that, 2^-11 of f16 and 2^-20 of the exponential. The output: the weights'
    errors over the largest value, above and below the line, then bf16's half
    unit, 2^-8."""
    ds = 2.0 ** -17 * reach
    dw = np.expm1(ds) + 2.0 ** -11 + 2.0 ** -20
    out = 2.0 ** -8 * np.abs(ref) + 2 * dw[..., None] * spread + 1e-30
    return out, ds + 2e-6 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))


def check_decode(got_out, got_lse, want, what=""):
    ref, lse, reach, spread = want
    out = got_out.float().cpu().numpy().astype(np.float64)
    glse = got_lse.cpu().numpy().astype(np.float64)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(out), nan), f"{what}: NaN positions"
    t_out, t_lse = tolerances(ref, reach, np.where(nan, 0.0, spread), lse)
    err = np.where(nan, 0.0, np.abs(out - ref))
    assert (err <= np.where(nan, 1.0, t_out)).all(), f"{what}: {np.nanmax(err / t_out)} of the tolerance"
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(glse), empty), f"{what}: empty rows"
    assert (out[empty] == 0).all(), f"{what}: empty rows are zeros"
    fin = np.isfinite(lse)
    assert np.array_equal(np.isfinite(glse), fin)
    assert (np.abs(glse[fin] - lse[fin]) <= t_lse[fin]).all(), f"{what}: lse"


def in_a_fresh_process(code):
    """Runs `code` where nothing has called the library yet."""
    path = os.pathsep.join([os.path.dirname(TESTS), TESTS])
    r = subprocess.run([sys.executable, "-c", code], cwd=TESTS, env={**os.environ, "PYTHONPATH": path},
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
