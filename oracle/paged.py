"""CPU oracle of the paged-cache calls, in 64 bits and from their definitions
(include/smd.h); shares no code with the GPU path. numpy only; used by the
tests."""
from __future__ import annotations

import math

import numpy as np

MIN_EXPONENT = -120
BF16_MAX = float(np.array(0x7f7f0000, dtype=np.uint32).view(np.float32))


def e4m3_values() -> np.ndarray:
    """The 256 values of E4M3: 1.4.3 bits, exponent bias 7, no infinities."""
    v = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if (code & 127) == 127:
            x = math.nan
        v[code] = -x if code & 128 else x
    return v


VALUES = e4m3_values()


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Codes nearest to x, ties to the even code, saturating; NaN to 0x7f."""
    grid = VALUES[:127]
    a = np.minimum(np.abs(x), 448.0)
    nan = np.isnan(a)
    a = np.where(nan, 0.0, a)
    below = np.clip(np.searchsorted(grid, a, side="right") - 1, 0, 126)
    above = np.minimum(below + 1, 126)
    down, up = a - grid[below], grid[above] - a
    code = np.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    return np.where(nan, 127, code + 128 * np.signbit(x)).astype(np.uint8)


def bf16_round(x: np.ndarray) -> np.ndarray:
    """float64 values of the bf16 nearest to x (through fp32; ties to even)."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = (u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000
    out = r.astype(np.uint32).view(np.float32).astype(np.float64)
    return np.where(np.isnan(x), np.nan, out)


def block_tables(lengths, new_tokens, table, ring, state, P, T):
    """(new_lengths, new_state, starts, slots, positions, table, ring, refused), request by request."""
    table, ring = table.copy(), ring.copy()
    R, W = table.shape
    N = len(ring)
    taken, given = int(state[0]), int(state[1])
    free = given - taken
    new_lengths, starts, slots, positions = [], [0], [], []
    needs = tokens = used = 0
    back, refused = given, False
    source = ring.copy()
    for r in range(R):
        length = min(max(int(lengths[r]), 0), W * P)
        n = int(new_tokens[r])
        have = -(-length // P)
        if n < 0:
            for j in range(have):
                ring[back % N] = table[r, j]
                back += 1
            new_lengths.append(0)
            starts.append(starts[-1])
            continue
        total = -(-(length + n) // P)
        if total > W:
            refused, ok = True, n == 0
        else:
            at, need = needs, total - have
            needs += need
            ok = need == 0 or needs <= free
            if ok:
                tokens += n
                ok = n == 0 or tokens <= T
            refused = refused or not ok
            if ok:
                for j in range(need):
                    table[r, have + j] = source[(taken + at + j) % N]
                used += need
        g = n if ok else 0
        for p in range(length, length + g):
            slots.append(int(table[r, p // P]) * P + p % P)
            positions.append(p)
        new_lengths.append(length + g)
        starts.append(starts[-1] + g)
    slots += [-1] * (T - len(slots))
    positions += [-1] * (T - len(positions))
    return (np.array(new_lengths), np.array([taken + used, back]), np.array(starts), np.array(slots),
            np.array(positions), table, ring, refused)


def power(a: float) -> float:
    """The least power of two at which a / 2^e is at most 448."""
    if a == 0.0:
        return 2.0 ** MIN_EXPONENT
    e = math.floor(math.log2(a / 448.0)) - 1
    while a / 2.0 ** e > 448.0:
        e += 1
    return 2.0 ** max(e, MIN_EXPONENT)


def paged_append(pools, scales, bounds, x, slots):
    """Writes tokens into codes pools[side][page, head, token, column] (uint8),
    scales[side][page, head] and bounds [page, head, 2, column] (float64), in place.
    x[side]: [T, heads, columns] values."""
    pages, heads, P, _ = pools[0].shape
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if s < 0 or s // P >= pages:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) % P != 0:
            n += 1
        page, o = s // P, s % P
        for side in (0, 1):
            for h in range(heads):
                given = x[side][t:t + n, h]
                y = np.clip(given, -BF16_MAX, BF16_MAX)
                a = np.nanmax(np.abs(y)) if not np.isnan(y).all() else 0.0
                scale = power(float(a))
                if o:
                    old = float(scales[side][page, h])
                    scale = max(scale, old)
                    kept = VALUES[pools[side][page, h, :o]]
                    pools[side][page, h, :o] = e4m3_encode(kept * old / scale)
                pools[side][page, h, o:o + n] = e4m3_encode(given / scale)  # infinities saturate
                scales[side][page, h] = scale
                if side == 0 and bounds is not None:
                    hi = np.fmax.reduce(y, axis=0, initial=-np.inf)
                    lo = np.fmin.reduce(y, axis=0, initial=np.inf)
                    if o:
                        hi = np.maximum(hi, bounds[page, h, 0])
                        lo = np.minimum(lo, bounds[page, h, 1])
                    bounds[page, h, 0] = np.clip(hi, -BF16_MAX, BF16_MAX)
                    bounds[page, h, 1] = np.clip(lo, -BF16_MAX, BF16_MAX)
        t += n


def row_limit(length: int, i: int, G: int) -> int:
    return max(length - G + 1 + i, 0)


def block_scores(q, bounds, table, lengths, P, G, keep_first=0, keep_last=0):
    """[B, heads, width] scores before rounding; +inf where kept, NaN past a row's pages."""
    B, Hq, D = q.shape
    heads = bounds.shape[1]
    g = Hq // heads
    W = table.shape[1]
    out = np.full((B, heads, W), np.nan)
    for b in range(B):
        r, i = divmod(b, G)
        n = min(max(int(lengths[r]), 0), W * P)
        sees = -(-row_limit(n, i, G) // P)
        for j in range(sees):
            p = int(table[r, j])
            for h in range(heads):
                hi, lo = bounds[p, h] if 0 <= p < len(bounds) else np.zeros((2, D))
                rows = q[b, h * g:(h + 1) * g]
                out[b, h, j] = np.maximum(rows * hi, rows * lo).sum(1).max()
        out[b, :, :min(keep_first, sees)] = np.inf
        out[b, :, max(sees - keep_last, 0):sees] = np.inf
    return out


def paged_decode(q, pools, scales, table, lengths, sm_scale, G=1, lists=None, counts=None):
    """(out, lse, reach, spread): reach[b, a] is the largest sm_scale * sum_c |q_c k_c|
    over the tokens seen (the size that fp32 sums of the logits round at), and
    spread the largest |v| of each column."""
    B, Hq, D = q.shape
    pages, heads, P, _ = pools[0].shape
    g, W = Hq // heads, table.shape[1]
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    reach, spread = np.zeros((B, Hq)), np.zeros((B, Hq, D))
    for b in range(B):
        r, i = divmod(b, G)
        lim = row_limit(min(max(int(lengths[r]), 0), W * P), i, G)
        for h in range(heads):
            if lists is None:
                blocks = range(-(-lim // P))
            else:
                c = lists.shape[2] if counts is None else min(max(int(counts[b, h]), 0), lists.shape[2])
                blocks = [int(j) for j in lists[b, h, :c]]
            ks, vs = [], []
            for j in blocks:
                if j < 0 or j * P >= lim:
                    continue
                n, p = min(P, lim - j * P), int(table[r, j])
                if 0 <= p < pages:
                    ks.append(VALUES[pools[0][p, h, :n]] * float(scales[0][p, h]))
                    vs.append(VALUES[pools[1][p, h, :n]] * float(scales[1][p, h]))
                else:
                    ks.append(np.zeros((n, D)))
                    vs.append(np.zeros((n, D)))
            if not ks:
                continue
            k, v = np.concatenate(ks), np.concatenate(vs)
            for a in range(h * g, (h + 1) * g):
                s = sm_scale * (k @ q[b, a])
                m = s.max()
                w = np.exp(s - m)
                out[b, a] = w @ v / w.sum()
                lse[b, a] = m + math.log(w.sum())
                reach[b, a] = sm_scale * (np.abs(k) @ np.abs(q[b, a])).max()
                spread[b, a] = np.abs(v).max(0)
    return out, lse, reach, spread
