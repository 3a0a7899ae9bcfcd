"""CPU oracle of the calls on the 4-bit cache and the step around it, in 64 bits or
whole numbers and from their definitions (include/smd.h); shares no code with the GPU
path. numpy only; used by the tests."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from . import paged as opaged

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])  # of the E2M1 codes 0 to 7
VALUES = np.concatenate([GRID, -GRID])


def e2m1_encode(x: np.ndarray) -> np.ndarray:
    """Codes nearest to x, ties to the even code, saturating; NaN as 0."""
    a = np.minimum(np.nan_to_num(np.abs(x), nan=0.0, posinf=6.0), 6.0)
    below = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 7)
    above = np.minimum(below + 1, 7)
    down, up = a - GRID[below], GRID[above] - a
    code = np.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    return (code + 8 * (np.signbit(x) & (code > 0))).astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def values(packed, scales, exps=None) -> np.ndarray:
    """[pages, heads, tokens, columns] values of a pool."""
    v = VALUES[unpack(packed)].reshape(*packed.shape[:-1], -1, 16) * opaged.VALUES[scales][..., None]
    v = v.reshape(*packed.shape[:-1], -1)
    if exps is not None:
        v = v * np.exp2(np.clip(np.asarray(exps, dtype=np.float64), -100, 100))[:, None, None]
    return v


def quantise(x, exps):
    """Packed codes and scales of x [tokens, heads, columns]; exps [heads]."""
    with np.errstate(invalid="ignore", over="ignore"):
        y = x * np.exp2(-np.clip(np.asarray(exps, dtype=np.float64), -100, 100))[:, None]
        y = y.reshape(*x.shape[:2], -1, 16)
        s = opaged.e4m3_encode(np.abs(y).max(-1) / 6)  # max: a NaN stays one
        sv = opaged.VALUES[s][..., None]
        z = np.where(sv > 0, y / np.where(sv > 0, sv, 1.0), 0.0)
    return pack(e2m1_encode(z).reshape(x.shape)), s


def paged4_append(pools, scales, exps, bounds, x, slots):
    """Writes tokens into pools[side] [pages, heads, P, D / 2], scales[side] and bounds
    [page, head, 2, column] (float64), in place. x[side]: [T, heads, columns]."""
    pages, heads, P, _ = pools[0].shape
    for side in (0, 1):
        codes, s = quantise(x[side], exps[side] if exps[side] is not None else np.zeros(heads))
        for t, slot in enumerate(slots):
            if 0 <= slot and slot // P < pages:
                pools[side][slot // P, :, slot % P] = codes[t]
                scales[side][slot // P, :, slot % P] = s[t]
    if bounds is None:
        return
    y = np.clip(x[0], -opaged.BF16_MAX, opaged.BF16_MAX)
    t = 0
    while t < len(slots):
        s, n = int(slots[t]), 1
        if s < 0 or s // P >= pages:
            t += 1
            continue
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) % P != 0:
            n += 1
        hi = np.fmax.reduce(y[t:t + n], axis=0, initial=-np.inf)
        lo = np.fmin.reduce(y[t:t + n], axis=0, initial=np.inf)
        if s % P:
            hi, lo = np.maximum(hi, bounds[s // P, :, 0]), np.minimum(lo, bounds[s // P, :, 1])
        bounds[s // P, :, 0] = np.clip(hi, -opaged.BF16_MAX, opaged.BF16_MAX)
        bounds[s // P, :, 1] = np.clip(lo, -opaged.BF16_MAX, opaged.BF16_MAX)
        t += n


def attend(q, k, v, table, lengths, sm_scale, G=1, lists=None, counts=None):
    """(out, lse, reach, spread) as the E4M3 cache's oracle gives them, of pools' values k
    and v [pages, heads, P, D]."""
    B, Hq, D = q.shape
    pages, heads, P, _ = k.shape
    g, W = Hq // heads, table.shape[1]
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    reach, spread = np.zeros((B, Hq)), np.zeros((B, Hq, D))
    for b in range(B):
        r, i = divmod(b, G)
        lim = max(min(max(int(lengths[r]), 0), W * P) - G + 1 + i, 0)
        for h in range(heads):
            if lists is None:
                blocks = range(-(-lim // P))
            else:
                c = lists.shape[2] if counts is None else min(max(int(counts[b, h]), 0), lists.shape[2])
                blocks = [int(j) for j in lists[b, h, :c] if 0 <= j and j * P < lim]
            ks, vs = [], []
            for j in blocks:
                n, p = min(P, lim - j * P), int(table[r, j])
                inside = 0 <= p < pages
                ks.append(k[p, h, :n] if inside else np.zeros((n, D)))
                vs.append(v[p, h, :n] if inside else np.zeros((n, D)))
            if not ks:
                continue
            kk, vv = np.concatenate(ks), np.concatenate(vs)
            for a in range(h * g, (h + 1) * g):
                s = sm_scale * (kk @ q[b, a])
                m = s.max()
                w = np.exp(s - m)
                out[b, a] = w @ vv / w.sum()
                lse[b, a] = m + np.log(w.sum())
                reach[b, a] = abs(sm_scale) * (np.abs(kk) @ np.abs(q[b, a])).max()
                spread[b, a] = np.abs(vv).max(0)
    return out, lse, reach, spread


def qk_norm_rope(x, weight, eps, positions, freqs, interleaved):
    """(y, reach): one side's heads [T, H, D] in 64 bits; reach: for each element the size of what
    its rotation adds up. positions [axes, T], freqs [axes, rot / 2], or None."""
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    reach = np.abs(y)
    if positions is None:
        return y, reach
    half = freqs.shape[1]
    # The angle modulo a turn, from whole numbers: a frequency is a fraction of powers of two.
    angle = np.zeros((x.shape[0], half))
    for j in range(half):
        f = [Fraction(float(v)) for v in freqs[:, j]]
        for t in range(x.shape[0]):
            whole = sum(int(p) * v for p, v in zip(positions[:, t], f))
            angle[t, j] = _reduced(whole)
    u = np.arange(half) * (2 if interleaved else 1)
    v = u + (1 if interleaved else half)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = y[..., u], y[..., v]
    out = y.copy()
    out[..., u], out[..., v] = a * c - b * s, a * s + b * c
    reach[..., u] = reach[..., v] = np.abs(a) + np.abs(b)
    return out, reach


# pi to 50 digits, as a fraction.
_PI = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


def _reduced(x: Fraction) -> float:
    turns = x / (2 * _PI)
    return float((turns - round(turns)) * 2 * _PI)


def verify_drafts(target, draft, tokens, accept, sample):
    """(out_tokens, accepted, rejected), in whole numbers and fractions. Probabilities float32."""
    R, G, V = target.shape
    out = np.full((R, G), -1, dtype=np.int64)
    stay = np.zeros(R, dtype=np.int64)

    def share(x):
        x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(0), np.float32(1)))
        return [int(w) for w in np.floor(x.astype(np.float64) * 2.0 ** 40)]

    for r in range(R):
        a, refused = 0, False
        while a < G - 1:
            d = int(tokens[r, a])
            if not 0 <= d < V:
                break
            p, u = float(target[r, a, d]), float(accept[r, a])
            q = 1.0 if draft is None else float(draft[r, a, d])
            if math.isnan(p) or math.isnan(q) or math.isnan(u):
                refused = True
            elif all(map(math.isfinite, (p, q, u))):
                refused = not Fraction(u) * Fraction(q) < Fraction(p)
            else:
                refused = not u * q < p
            if refused:
                break
            a += 1
        stay[r] = a
        out[r, :a] = tokens[r, :a]
        row = target[r, a]
        if refused:
            with np.errstate(invalid="ignore"):
                left = row.copy() if draft is None else row - draft[r, a]
            if draft is None:
                left[int(tokens[r, a])] = 0
        else:
            left = row
        w = share(left)
        if sum(w) == 0:
            w = share(row)
        total = sum(w)
        if total == 0:
            continue
        u = float(sample[r])
        U = 0 if math.isnan(u) else min(max(math.floor(u * 2.0 ** 31) if math.isfinite(u) else
                                            (2 ** 31 if u > 0 else 0), 0), 2 ** 31 - 1)
        t, run = U * total >> 31, 0
        for v, x in enumerate(w):
            run += x
            if run > t:
                out[r, a] = v
                break
    return out, stay, G - 1 - stay


def block_trim(lengths, drop, table, ring, state, P):
    """(new_lengths, new_state, ring), request by request."""
    ring = ring.copy()
    W, N = table.shape[1], len(ring)
    taken, given = int(state[0]), int(state[1])
    new = []
    for r in range(len(lengths)):
        length = min(max(int(lengths[r]), 0), W * P)
        left = max(length - max(int(drop[r]), 0), 0)
        for j in range(-(-left // P), -(-length // P)):
            ring[given % N] = table[r, j]
            given += 1
        new.append(left)
    return np.array(new), np.array([taken, given]), ring
